"""Tree attention over the 8-bit paged cache against 64 bits, element by element (the bound is derived in
kv8_helpers), its refusals on the device, and that what a row does not see has no influence on it."""

import numpy as np
import pytest
import torch

import tree_speculative_decoding_split_gb300 as st
from gen import trees as T
import kv8_helpers as K8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("G,Hkv,bs", [(4, 2, 64), (1, 1, 16), (8, 1, 32), (5, 2, 128), (16, 1, 256)])
def test_single_tokens(d, G, Hkv, bs):
    """Lengths from none to several splits, ends inside and at the end of boxes, blocks and splits."""
    rng = np.random.default_rng(d + G)
    lens = [0, 1, 15, 16, 17, 63, 64, 65, 255, 256, 257, 511, 777, 1500]
    cache = K8.Cache(rng, lens, Hkv, d, bs, max_len=2000)
    qs = K8.Queries(rng, len(lens), 1, G * Hkv, Hkv, d)
    out, lse, status = K8.attend(K8.dev(), cache, qs)
    assert status == 0
    K8.check(cache, qs, out, lse)


@pytest.mark.parametrize("N,G,Hkv,d,bs,lens", [
    (2, 4, 2, 128, 64, [100, 0, 300]), (4, 4, 1, 128, 16, [1000, 31]), (7, 2, 2, 64, 32, [129, 700]),
    (17, 1, 2, 128, 64, [64, 65, 1]), (33, 3, 1, 128, 128, [500, 127]), (63, 4, 2, 128, 16, [777, 3, 0]),
    (63, 8, 1, 64, 64, [300, 2100]), (127, 2, 1, 128, 256, [400, 1030]), (255, 1, 2, 128, 32, [0, 250]),
    (255, 8, 1, 128, 64, [1300]), (255, 5, 1, 64, 16, [129])])
def test_trees(N, G, Hkv, d, bs, lens):
    rng = np.random.default_rng(N * G + d)
    cache = K8.Cache(rng, lens, Hkv, d, bs, max_len=max(lens) + 500)
    nn = [max(1, N - 5 * b) for b in range(len(lens))]
    qs = K8.Queries(rng, len(lens), N, G * Hkv, Hkv, d, n_nodes=nn)
    out, lse, status = K8.attend(K8.dev(), cache, qs)
    assert status == 0
    K8.check(cache, qs, out, lse)


def test_long_prefix_and_chain():
    rng = np.random.default_rng(3)
    cache = K8.Cache(rng, [9000, 5], 1, 128, 16)
    qs = K8.Queries(rng, 2, 40, 4, 1, 128, parents=[T.chain_tree(40)] * 2)
    out, lse, status = K8.attend(K8.dev(), cache, qs)
    assert status == 0
    K8.check(cache, qs, out, lse)


@pytest.mark.parametrize("N,G,B,long", [(1, 4, 20, 30000), (1, 8, 150, 20000), (1, 1, 130, 0), (3, 5, 40, 9001),
                                        (63, 4, 12, 12000), (40, 8, 140, 6001), (255, 4, 3, 5000), (20, 1, 129, 0)])
def test_one_long_request_among_many(N, G, B, long):
    """Ragged batches, where the long prefix takes most of the splits; the last request is longer than its table."""
    rng = np.random.default_rng(B + N)
    lens = [int(x) for x in rng.integers(0, 90, B)]
    lens[1] = 1500
    lens[B // 2] = long
    cache = K8.Cache(rng, lens, 1, 128, 64, max_len=max(lens) + 64)
    qs = K8.Queries(rng, B, N, G, 1, 128)
    out, lse, status = K8.attend(K8.dev(), _with_lens(cache, lens[:-1] + [10 ** 8]), qs)
    assert status == 7
    assert not out[-1].any() and not lse[-1].any()
    K8.check(cache, qs, out, lse, requests=sorted({0, 1, B // 2, B - 2}))


@pytest.mark.parametrize("N", [1, 40])
def test_any_scale_and_softmax_scale(N):
    """Scales that are no powers of two, far apart (2^-20 to 2^20), and a softmax scale of the caller's."""
    rng = np.random.default_rng(4)
    cache = K8.Cache(rng, [400, 90], 2, 128, 16, pow2=False, scale_spread=0)
    cache.vs *= 2.0 ** rng.integers(-20, 21, cache.vs.shape).astype(np.float32)
    cache.ks *= 2.0 ** rng.integers(-3, 3, cache.ks.shape).astype(np.float32)
    qs = K8.Queries(rng, 2, N, 8, 2, 128)
    out, lse, status = K8.attend(K8.dev(), cache, qs, scale=0.03)
    assert status == 0
    K8.check(cache, qs, out, lse, scale=0.03)


@pytest.mark.parametrize("N", [1, 3, 60])
@pytest.mark.parametrize("e", [-50, -30, 100])
def test_values_far_from_one(N, e):
    """All of V near 2^e, in the cache and in the tree: the weights keep their precision whatever V's unit."""
    rng = np.random.default_rng(11)
    cache = K8.Cache(rng, [300, 47], 1, 128, 32)
    qs = K8.Queries(rng, 2, N, 4, 1, 128)
    cache.vs *= np.float32(2.0 ** e)
    qs.vt_t = qs.vt_t * 2.0 ** e
    qs.vt = qs.vt_t.double().numpy()
    out, lse, status = K8.attend(K8.dev(), cache, qs)
    assert status == 0
    K8.check(cache, qs, out, lse)


@pytest.mark.parametrize("N", [1, 60])
def test_sharp_and_flat_rows(N):
    """Scores hundreds apart (one key takes all) and queries of zeros (every key the same)."""
    rng = np.random.default_rng(5)
    cache = K8.Cache(rng, [600, 130], 1, 128, 64)
    qs = K8.Queries(rng, 2, N, 4, 1, 128, spread=30.0)
    qs.q_t[:, :, 0] = 0
    qs.q = qs.q_t.double().numpy()
    out, lse, status = K8.attend(K8.dev(), cache, qs)
    assert status == 0
    K8.check(cache, qs, out, lse)


@pytest.mark.parametrize("N,G", [(9, 1), (40, 4), (255, 8)])
def test_unseen_rows_have_no_influence(N, G):
    """Infinities and NaN in K/V of nodes outside a row's path, and in padded nodes, change nothing; a
    row that sees an infinity in V gets it."""
    dev = K8.dev()
    rng = np.random.default_rng(6 + N)
    cache = K8.Cache(rng, [200, 70], 1, 128, 64)
    nn = [N, N - 3]
    qs = K8.Queries(rng, 2, N, G, 1, 128, n_nodes=nn)
    clean, clean_lse, _ = K8.attend(dev, cache, qs)
    leaf = N // 2
    see = np.array([[leaf in _path(qs.parent[b], i) if i < nn[b] else False for i in range(N)] for b in range(2)])
    qs.kt_t[1, nn[1]:] = float("nan")
    qs.vt_t[1, nn[1]:] = float("inf")
    qs.vt_t[:, leaf, 0, 7] = float("inf")
    qs.vt_t[:, leaf, 0, 100] = float("nan")
    out, lse, status = K8.attend(dev, cache, qs)
    assert status == 0
    assert np.array_equal(out[~see], clean[~see]) and np.array_equal(lse, clean_lse)
    assert see.any() and np.isposinf(out[see][..., 7]).all() and np.isnan(out[see][..., 100]).all()
    rest = np.ones(128, bool)
    rest[[7, 100]] = False
    assert np.array_equal(out[see][..., rest], clean[see][..., rest])
    qs.kt_t[:, leaf] = float("nan")
    out, lse, status = K8.attend(dev, cache, qs)
    assert np.array_equal(out[~see], clean[~see]) and np.array_equal(lse[~see], clean_lse[~see])
    assert np.isnan(out[see]).all()


def _path(parent, i):
    path = []
    while i >= 0:
        path.append(i)
        i = int(parent[i])
    return path


@pytest.mark.parametrize("N", [1, 50])
def test_bad_requests_are_zeroed_alone(N):
    dev = K8.dev()
    rng = np.random.default_rng(7)
    lens = [500, 300, 3000, 40, 90, 800]
    for kind, code in (("table", 7), ("table_late", 7), ("len", 7), ("tree", 4), ("count", 4)):
        cache = K8.Cache(rng, lens, 2, 128, 32, max_len=3100)
        qs = K8.Queries(rng, len(lens), N, 4, 2, 128)
        given = list(lens)
        if kind == "table":
            cache.table[1, 2] = cache.k.shape[0]
        if kind == "table_late":
            cache.table[1, 9] = -1
        if kind == "len":
            given[1] = cache.max_blocks * 32 + 1
        if kind == "tree":
            qs.parent[1, 0] = 0
        if kind == "count":
            qs.n_nodes[1] = 0
        out, lse, status = K8.attend(dev, _with_lens(cache, given), qs)
        assert status == code, kind
        assert (out[1] == 0).all() and (lse[1] == 0).all(), kind
        K8.check(cache, qs, out, lse, requests=[0, 2, 3, 4, 5])


def _with_lens(cache, lens):
    import copy
    c = copy.copy(cache)
    c.lens = lens
    return c


def test_entries_behind_the_prefix_are_not_read():
    """Table entries past the last block of the prefix may be anything."""
    rng = np.random.default_rng(8)
    cache = K8.Cache(rng, [100, 64], 1, 64, 16, max_len=400)
    cache.table[cache.table < 0] = 1 << 30
    qs = K8.Queries(rng, 2, 3, 2, 1, 64)
    out, lse, status = K8.attend(K8.dev(), cache, qs)
    assert status == 0
    K8.check(cache, qs, out, lse)


@pytest.mark.parametrize("N", [1, 63])
def test_blocks_beyond_two_gigabytes(N):
    """Blocks whose byte offset in the pool passes 2^31."""
    dev = K8.dev()
    rng = np.random.default_rng(9)
    cache = K8.Cache(rng, [700, 300], 8, 128, 256)
    small = cache.device(dev)
    nb = 8700
    at = nb - cache.k.shape[0]
    big = {}
    for name in ("k_cache", "v_cache"):
        pool = torch.zeros((nb, 8, 256, 128), dtype=torch.uint8, device=dev)
        pool[at:] = small[name].view(torch.uint8)
        big[name] = pool.view(torch.float8_e4m3fn)
    for name in ("k_scale", "v_scale"):
        big[name] = torch.ones((nb, 8), device=dev)
        big[name][at:] = small[name]
    big["block_table"] = torch.where(small["block_table"] >= 0, small["block_table"] + at, small["block_table"])
    qs = K8.Queries(rng, 2, N, 16, 8, 128)
    lens = torch.tensor(cache.lens, dtype=torch.int32, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    out, lse = st.tree_attention_kv8(qs.q_t.to(dev), qs.kt_t.to(dev), qs.vt_t.to(dev), big["k_cache"], big["v_cache"],
                                     big["k_scale"], big["v_scale"], lens, torch.from_numpy(qs.n_nodes).to(dev),
                                     torch.from_numpy(qs.parent).to(dev), big["block_table"], dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    K8.check(cache, qs, out.double().cpu().numpy(), lse.double().cpu().numpy())


@pytest.mark.parametrize("N", [1, 30])
def test_repeats_and_streams_agree_to_the_bit(N):
    """The same call again, on another stream with a workspace of the caller's, and with other requests
    around it: the same bits."""
    dev = K8.dev()
    rng = np.random.default_rng(10)
    cache = K8.Cache(rng, [1200, 37, 600], 2, 128, 64)
    qs = K8.Queries(rng, 3, N, 8, 2, 128)
    out, lse, _ = K8.attend(dev, cache, qs)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    again, lse2, _ = K8.attend(dev, cache, qs, stream=side)
    assert np.array_equal(out, again) and np.array_equal(lse, lse2)
    with torch.cuda.stream(side):
        ws = torch.full((1 << 26,), 0xFF, dtype=torch.uint8, device=dev)  # NaN bytes: nothing of it may be read unwritten
        again, lse2, _ = K8.attend(dev, cache, qs, workspace=ws)
    assert np.array_equal(out, again) and np.array_equal(lse, lse2)


@pytest.mark.parametrize("N", [1, 40])
def test_calls_on_two_streams_at_once(N):
    dev = K8.dev()
    rng = np.random.default_rng(12)
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    calls, want = [], []
    for i in range(2):
        cache = K8.Cache(rng, [3000 + i, 200, 900], 2, 128, 32)
        qs = K8.Queries(rng, 3, N, 8, 2, 128)
        out, lse, status = K8.attend(dev, cache, qs)
        assert status == 0
        c = cache.device(dev)
        lens = torch.tensor(cache.lens, dtype=torch.int32, device=dev)
        rest = [torch.from_numpy(x).to(dev) for x in (qs.n_nodes, qs.parent)]
        calls.append((qs.q_t.to(dev), qs.kt_t.to(dev), qs.vt_t.to(dev), c["k_cache"], c["v_cache"], c["k_scale"],
                      c["v_scale"], lens, *rest, c["block_table"]))
        want.append(torch.from_numpy(out))
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, side in enumerate(sides):
            got[i].append(st.tree_attention_kv8(*calls[i], stream=side)[0])
    torch.cuda.synchronize()
    for i in range(2):
        for out in got[i]:
            assert torch.equal(out.double().cpu(), want[i])
