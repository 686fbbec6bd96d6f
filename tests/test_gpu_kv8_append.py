"""Appending rows to the 8-bit paged cache: codes and scales bit for bit against the oracle."""

import numpy as np
import pytest
import torch

import oracle
import tree_speculative_decoding_split_gb300 as st
from gen import trees as T
import kv8_helpers as K8

pytestmark = pytest.mark.gpu


def _rows(rng, shape, dtype, grow):
    x = rng.standard_normal(shape) * 2.0 ** rng.integers(-4, grow, shape[:1] + (1,) * (len(shape) - 1))
    t = torch.from_numpy(x.astype(np.float32)).to(dtype)
    return t, t.double().numpy()


def _device(cache, dev):
    c = cache.device(dev)
    return c, dict(k_cache=c["k_cache"], v_cache=c["v_cache"], k_scale=c["k_scale"], v_scale=c["v_scale"],
                   block_table=c["block_table"])


def _compare(cache, c):
    torch.cuda.synchronize()
    for codes, scale, name in ((cache.k, cache.ks, "k"), (cache.v, cache.vs, "v")):
        assert np.array_equal(c[name + "_scale"].cpu().numpy(), scale.astype(np.float32)), name
        got = c[name + "_cache"].view(torch.uint8).cpu().numpy()
        same = (got == codes) | (np.isnan(oracle.E4M3[got]) & np.isnan(oracle.E4M3[codes]))
        assert same.all(), (name, np.argwhere(~same)[:4].tolist())


def _oracle_append(cache, b, rows_k, rows_v, start):
    ks, vs = cache.ks.astype(np.float64), cache.vs.astype(np.float64)
    oracle.append_rows(rows_k, cache.k, ks, start, cache.table[b], cache.bs)
    oracle.append_rows(rows_v, cache.v, vs, start, cache.table[b], cache.bs)
    cache.ks, cache.vs = ks, vs


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("bs,Hkv,d", [(16, 1, 64), (16, 3, 128), (32, 2, 64), (64, 8, 128), (128, 2, 128), (256, 2, 64),
                                      (256, 5, 128)])
def test_packed_rows(dtype, bs, Hkv, d):
    dev = K8.dev()
    rng = np.random.default_rng(bs + d)
    start = [0, 5, bs, 2 * bs - 1, 7, 3, 0, 3 * bs + 2]
    add = [3 * bs + 1, bs - 5, 1, 2, 0, 2 * bs, bs, 1]
    cache = K8.Cache(rng, [a + n for a, n in zip(start, add)], Hkv, d, bs)
    c, kw = _device(cache, dev)
    rk, k = _rows(rng, (sum(add), Hkv, d), dtype, 7)
    rv, v = _rows(rng, (sum(add), Hkv, d), dtype, 7)
    rs = np.concatenate([[0], np.cumsum(add)]).astype(np.int32)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    new = st.kv8_append(rk.to(dev), rv.to(dev), seq_len=torch.tensor(start, dtype=torch.int32, device=dev),
                        row_start=torch.from_numpy(rs).to(dev), dev_status=status, **kw)
    for b in range(len(add)):
        _oracle_append(cache, b, k[rs[b]: rs[b + 1]], v[rs[b]: rs[b + 1]], start[b])
    _compare(cache, c)
    assert int(status.item()) == 0 and new.tolist() == [a + n for a, n in zip(start, add)]


@pytest.mark.parametrize("dtype,N,bs,d", [(torch.bfloat16, 63, 16, 128), (torch.bfloat16, 255, 64, 64),
                                          (torch.float32, 40, 32, 128), (torch.bfloat16, 1, 256, 128)])
def test_accepted_paths(dtype, N, bs, d):
    dev = K8.dev()
    rng = np.random.default_rng(N + bs)
    B, Hkv = 7, 2
    start = [0, 1, bs - 1, bs, 5 * bs - 2, 33, 2 * bs + 3]
    parents = [T.random_bfs_tree(rng, N, 9)[0] for _ in range(B)]
    paths = []
    for b in range(B):
        i, p = int(rng.integers(0, N)), []
        while i >= 0:
            p.append(i)
            i = int(parents[b][i])
        paths.append(p[::-1])
    cap = max(len(p) for p in paths) + 1
    path = np.full((B, cap), -1, np.int32)
    for b, p in enumerate(paths):
        path[b, : len(p)] = p
    cache = K8.Cache(rng, [a + len(p) for a, p in zip(start, paths)], Hkv, d, bs)
    c, kw = _device(cache, dev)
    rk, k = _rows(rng, (B, N, Hkv, d), dtype, 7)
    rv, v = _rows(rng, (B, N, Hkv, d), dtype, 7)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    new = st.kv8_append(rk.to(dev), rv.to(dev), seq_len=torch.tensor(start, dtype=torch.int32, device=dev),
                        path=torch.from_numpy(path).to(dev),
                        accept_len=torch.tensor([len(p) - 1 for p in paths], dtype=torch.int32, device=dev),
                        dev_status=status, **kw)
    for b, p in enumerate(paths):
        _oracle_append(cache, b, k[b, p], v[b, p], start[b])
    _compare(cache, c)
    assert int(status.item()) == 0 and new.tolist() == [a + len(p) for a, p in zip(start, paths)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_extreme_values(dtype):
    """Zeros, the type's largest and smallest values, infinities and NaN; growth over a scale that is no
    power of two, down into subnormal codes, and one that stays."""
    dev = K8.dev()
    rng = np.random.default_rng(1)
    bs, Hkv, d = 16, 1, 64
    start = [0] * 6 + [8, 8, 8, 8]
    cache = K8.Cache(rng, [s + 4 for s in start], Hkv, d, bs, pow2=False)
    x = rng.standard_normal((len(start), 4, Hkv, d))
    x[0] = 0
    x[1, 0, 0, :3] = [3e38, -3e38, 1]
    x[2] = 1e-38
    x[2, 1] = 2.0 ** -130
    x[3, 1, 0, 5:9] = [np.inf, -np.inf, np.nan, 448]
    x[4] = np.nan
    x[5, :, :, 0] = np.float32(448 * 2.0 ** -64)
    x[6] *= 1000     # grows: the old codes shrink
    x[7] *= 1e-3     # the old scale stays
    x[8] *= 2e4      # old codes become subnormal
    x[9] = 0
    t = torch.from_numpy(x.astype(np.float32)).to(dtype)
    rows = t.double().numpy()
    c, kw = _device(cache, dev)
    flat = t.reshape(-1, Hkv, d).to(dev)
    rs = torch.arange(0, 4 * len(start) + 1, 4, dtype=torch.int32, device=dev)
    st.kv8_append(flat, flat.clone(), seq_len=torch.tensor(start, dtype=torch.int32, device=dev), row_start=rs, **kw)
    for b in range(len(start)):
        _oracle_append(cache, b, rows[b], rows[b], start[b])
    _compare(cache, c)


def test_appending_twice_is_the_same():
    """A call that is repeated with the same lengths writes the same codes (a replayed step)."""
    dev = K8.dev()
    rng = np.random.default_rng(2)
    cache = K8.Cache(rng, [40, 20], 2, 128, 16)
    c, kw = _device(cache, dev)
    rk, k = _rows(rng, (20, 2, 128), torch.bfloat16, 9)
    rs = torch.tensor([0, 12, 20], dtype=torch.int32, device=dev)
    args = dict(seq_len=torch.tensor([28, 12], dtype=torch.int32, device=dev), row_start=rs, **kw)
    st.kv8_append(rk.to(dev), rk.to(dev), **args)
    first = {n: c[n].view(torch.uint8).clone() if "cache" in n else c[n].clone() for n in c}
    st.kv8_append(rk.to(dev), rk.to(dev), **args)
    torch.cuda.synchronize()
    for n in c:
        assert torch.equal(c[n].view(torch.uint8) if "cache" in n else c[n], first[n]), n


@pytest.mark.parametrize("rows", [[0, 5, 4, 44], [0, 5, 200, 65], [0, 60, 10, 20], [-1, 5, 25, 65], [0, 5, 25, 66], [9, 8, 7, 6],
                                  [0, 1 << 30, -(1 << 31), 65]])
def test_rows_out_of_order_refuse_the_call(rows):
    """Nothing is written and no length moves, whichever request's range is the bad one."""
    dev = K8.dev()
    rng = np.random.default_rng(8)
    start = [3, 10, 0]
    cache = K8.Cache(rng, [48, 48, 48], 2, 64, 16)
    c, kw = _device(cache, dev)
    rk, _ = _rows(rng, (65, 2, 64), torch.bfloat16, 3)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    new = st.kv8_append(rk.to(dev), rk.to(dev), seq_len=torch.tensor(start, dtype=torch.int32, device=dev),
                        row_start=torch.tensor(rows, dtype=torch.int32, device=dev), dev_status=status, **kw)
    _compare(cache, c)
    assert int(status.item()) == 7 and new.tolist() == start


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("bs,d", [(16, 128), (64, 64), (128, 128), (256, 128), (256, 64)])
def test_tokens_and_a_prompt_in_one_call(dtype, bs, d):
    """One row for most requests, none for some, a prompt of several blocks for one: a block may have more new rows
    than the call's average suggests."""
    dev = K8.dev()
    rng = np.random.default_rng(bs * d)
    B, Hkv = 40, 3
    start = [int(x) for x in rng.integers(0, 2 * bs, B)]
    add = [1] * B
    add[3], add[7], add[20] = 0, 2 * bs + 5, 11
    cache = K8.Cache(rng, [a + n for a, n in zip(start, add)], Hkv, d, bs)
    c, kw = _device(cache, dev)
    rk, k = _rows(rng, (sum(add), Hkv, d), dtype, 7)
    rv, v = _rows(rng, (sum(add), Hkv, d), dtype, 7)
    rk[4, 1, 5] = float("inf")
    k[4, 1, 5] = np.inf
    rs = np.concatenate([[0], np.cumsum(add)]).astype(np.int32)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    new = st.kv8_append(rk.to(dev), rv.to(dev), seq_len=torch.tensor(start, dtype=torch.int32, device=dev),
                        row_start=torch.from_numpy(rs).to(dev), dev_status=status, **kw)
    for b in range(B):
        _oracle_append(cache, b, k[rs[b]: rs[b + 1]], v[rs[b]: rs[b + 1]], start[b])
    _compare(cache, c)
    assert int(status.item()) == 0 and new.tolist() == [a + n for a, n in zip(start, add)]


def test_rows_ahead_of_and_behind_the_requests():
    """Packed rows that belong to no request are not looked at."""
    dev = K8.dev()
    rng = np.random.default_rng(9)
    start, rs = [3, 17, 0], [70, 75, 75, 119]
    cache = K8.Cache(rng, [48, 48, 48], 2, 128, 16)
    c, kw = _device(cache, dev)
    rk, k = _rows(rng, (200, 2, 128), torch.bfloat16, 3)
    rk[:70] = float("nan")
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    new = st.kv8_append(rk.to(dev), rk.to(dev), seq_len=torch.tensor(start, dtype=torch.int32, device=dev),
                        row_start=torch.tensor(rs, dtype=torch.int32, device=dev), dev_status=status, **kw)
    for b in range(3):
        _oracle_append(cache, b, k[rs[b]: rs[b + 1]], k[rs[b]: rs[b + 1]], start[b])
    _compare(cache, c)
    assert int(status.item()) == 0 and new.tolist() == [8, 17, 44]


@pytest.mark.parametrize("kind,code", [("table", 7), ("len", 7), ("negative", 7)])
def test_bad_packed_requests(kind, code):
    dev = K8.dev()
    rng = np.random.default_rng(3)
    start, add = [3, 10, 0], [5, 20, 40]
    cache = K8.Cache(rng, [a + n for a, n in zip(start, add)], 2, 64, 16, max_len=48)
    rs = np.array([0, 5, 25, 65], np.int32)
    seq = list(start)
    if kind == "table":
        cache.table[1, 1] = cache.k.shape[0]
    if kind == "len":
        seq[1] = 29
    if kind == "negative":
        seq[1] = -1
    c, kw = _device(cache, dev)
    rk, k = _rows(rng, (65, 2, 64), torch.bfloat16, 3)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    new = st.kv8_append(rk.to(dev), rk.to(dev), seq_len=torch.tensor(seq, dtype=torch.int32, device=dev),
                        row_start=torch.from_numpy(rs).to(dev), dev_status=status, **kw)
    torch.cuda.synchronize()
    assert int(status.item()) == code
    assert new.tolist()[0] == start[0] + 5 and new.tolist()[1] == seq[1]
    _oracle_append(cache, 0, k[:5], k[:5], start[0])
    if kind in ("len", "negative"):
        _oracle_append(cache, 2, k[25:], k[25:], start[2])
    if kind == "table":  # the others as they should be; request 1's blocks are not compared
        _oracle_append(cache, 2, k[25:], k[25:], start[2])
        mine = [b for b in cache.table[0] if b >= 0] + [b for b in cache.table[2] if b >= 0]
        got = c["k_cache"].view(torch.uint8).cpu().numpy()
        for blk in mine:
            assert np.array_equal(got[blk] & 127 == 127, cache.k[blk] & 127 == 127)
            assert np.array_equal(np.nan_to_num(oracle.E4M3[got[blk]]), np.nan_to_num(oracle.E4M3[cache.k[blk]]))
    else:
        _compare(cache, c)


@pytest.mark.parametrize("kind,code", [("order", 4), ("root", 4), ("range", 4), ("long", 7), ("negative", 7), ("table", 7)])
def test_bad_paths_leave_the_request_alone(kind, code):
    dev = K8.dev()
    rng = np.random.default_rng(4)
    start = [14, 14]
    cache = K8.Cache(rng, [18, 18], 2, 128, 16)
    path = np.array([[0, 1, 3, -1], [0, 2, 4, -1]], np.int32)
    acc = np.array([2, 2], np.int32)
    if kind == "order":
        path[1, 2] = 2
    if kind == "root":
        path[1, 0] = 1
    if kind == "range":
        path[1, 2] = 6
    if kind == "long":
        acc[1] = 4
    if kind == "negative":
        acc[1] = -1
    if kind == "table":
        cache.table[1, 1] = -5
    c, kw = _device(cache, dev)
    rk, k = _rows(rng, (2, 6, 2, 128), torch.bfloat16, 9)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    new = st.kv8_append(rk.to(dev), rk.to(dev), seq_len=torch.tensor(start, dtype=torch.int32, device=dev),
                        path=torch.from_numpy(path).to(dev), accept_len=torch.from_numpy(acc).to(dev),
                        dev_status=status, **kw)
    _oracle_append(cache, 0, k[0, [0, 1, 3]], k[0, [0, 1, 3]], 14)
    _compare(cache, c)
    assert int(status.item()) == code and new.tolist() == [17, 14]


def test_no_rows():
    dev = K8.dev()
    cache = K8.Cache(np.random.default_rng(5), [20, 3], 1, 64, 16)
    c, kw = _device(cache, dev)
    empty = torch.empty((0, 1, 64), dtype=torch.bfloat16, device=dev)
    seq = torch.tensor([20, 3], dtype=torch.int32, device=dev)
    new = st.kv8_append(empty, empty, seq_len=seq, row_start=torch.zeros(3, dtype=torch.int32, device=dev), **kw)
    _compare(cache, c)
    assert new.tolist() == [20, 3]
