"""Tree attention over the 8-bit cache at the ends of what its inputs may hold: rows of zeros, rows next to bf16's
smallest and largest numbers, table entries out of range."""

import numpy as np
import pytest
import torch

import oracle
import tree_speculative_decoding_split_gb300 as st
import kv8_helpers as K8
import kv8_strict

pytestmark = pytest.mark.gpu

# (nodes, query heads per KV head, table slots): the few-rows kernel with one and two tiles of 8 rows, the tensor-core
# kernel with one group of 128 rows and, where the call is large enough by its table, with two
FORMS = [(1, 4, 600), (4, 4, 600), (20, 1, 600), (63, 4, 600), (40, 8, 10000)]


@pytest.mark.parametrize("N,G,slots", FORMS)
@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("bs", [16, 32, 64, 128])
def test_rows_of_zeros(N, G, slots, d, bs):
    """Every key weighs the same, whatever lies behind the prefix in its last block, box and tile, also where a
    block's keys are all zeros (its scale is then 2^-64)."""
    rng = np.random.default_rng(N + bs + d)
    lens = [1, 2, 65, 128, 129, 130, 193, 258, 514]
    cache = K8.Cache(rng, lens, 2, d, bs, max_len=slots)
    for b in (3, 4, 6, 8):
        blk = cache.table[b, (lens[b] - 1) // bs]
        cache.k[blk, :, : (lens[b] - 1) % bs + 1] = 0
        cache.ks[blk] = 2.0 ** -64
    qs = K8.Queries(rng, len(lens), N, 2 * G, 2, d)
    qs.q_t[:, :, 0] = 0
    qs.q_t[:, ::3, G] = 0
    qs.q_t[:, :, -1] = qs.q_t[:, :, -1] * 2.0 ** -125
    qs.q = qs.q_t.double().numpy()
    out, lse, status = K8.attend(K8.dev(), cache, qs)
    assert status == 0
    assert np.isfinite(out).all() and np.isfinite(lse).all()
    kv8_strict.check(cache, qs, out, lse)


@pytest.mark.parametrize("N,G,slots", FORMS)
@pytest.mark.parametrize("e,ke", [(22, 0), (27, 0), (31, 0), (60, 0), (104, 0), (120, 0), (126, -56), (127, -58), (20, 90)])
def test_large_queries(N, G, slots, e, ke):
    """Queries near 2^e and K scales near 2^ke, so that scores run from 2^26 to 2^124: one key takes a row's whole
    weight.  Request 0: a key each row points to.  Request 1: every score negative, the first key's least.

    The winner's score leads by more than half of itself, its error is 2^-13 of it at most (kv8_strict takes the
    same bound from kv8_helpers), so every other weight is 0 and the row is the winner's V row, which is exact in bf16."""
    rng = np.random.default_rng(N + e)
    d, lens = 128, [300, 3]
    cache = K8.Cache(rng, lens, 1, d, 64, max_len=slots)
    sign = rng.choice([-1.0, 1.0], (300, d))
    cache.k[cache.table[0, : 5]] = oracle.e4m3_encode(np.concatenate([sign * 64, np.zeros((20, d))]).reshape(5, 1, 64, d))
    cache.k[cache.table[1, 0], 0, :3] = oracle.e4m3_encode(sign[0] * np.array([[64], [104], [120]]))
    cache.ks[:] = 2.0 ** (ke - 6)
    qs = K8.Queries(rng, 2, N, G, 1, d)
    winner = rng.integers(0, 300, (N, G))
    qs.q_t, qs.q = K8.bf16(np.stack([sign[winner], np.broadcast_to(-sign[0], (N, G, d))]) *
                           rng.uniform(1, 1.9, (2, N, G, d)) * 2.0 ** e)
    qs.kt_t, qs.kt = K8.bf16(np.stack([rng.standard_normal((N, 1, d)) * 0.1, np.broadcast_to(sign[0] * 2, (N, 1, d))]) * 2.0 ** ke)
    out, lse, status = K8.attend(K8.dev(), cache, qs)
    assert status == 0
    v0, v1 = (cache.values(b)[1][0] for b in range(2))
    assert np.array_equal(out[0], v0[winner])
    assert np.array_equal(out[1], np.broadcast_to(v1[0], out[1].shape))
    kv8_strict.check(cache, qs, out, lse)


@pytest.mark.parametrize("N,G,slots", FORMS)
@pytest.mark.parametrize("e", [0, 30])
def test_rows_keep_their_bits_beside_large_ones(N, G, slots, e):
    """A head's rows are the same to the bit whatever the other heads' scores are."""
    rng = np.random.default_rng(N)
    cache = K8.Cache(rng, [300, 77], 1, 128, 64, max_len=slots)
    qs = K8.Queries(rng, 2, N, 2 * G, 1, 128)
    qs.q_t *= 2.0 ** e
    out, lse, _ = K8.attend(K8.dev(), cache, qs)
    qs.q_t[:, :, ::2] *= 2.0 ** 60
    again, lse2, status = K8.attend(K8.dev(), cache, qs)
    assert status == 0 and np.isfinite(again).all()
    assert np.array_equal(out[:, :, 1::2], again[:, :, 1::2]) and np.array_equal(lse[:, :, 1::2], lse2[:, :, 1::2])
    assert not np.array_equal(lse[:, :, ::2], lse2[:, :, ::2])


@pytest.mark.parametrize("N,G,slots", FORMS)
@pytest.mark.parametrize("e", range(24, 36))
def test_scores_a_few_steps_apart(N, G, slots, e):
    """Two keys whose scores, near 2^e in log2 units, differ by none to some float32 steps, the larger one later or in
    the tree: whichever weighs more, the row lies between their two V rows."""
    rng = np.random.default_rng(e)
    cache = K8.Cache(rng, [300, 130], 1, 128, 64, max_len=slots)
    cache.k[cache.table[0, :5]] = 0
    cache.k[cache.table[1, :3]] = 0
    one, two, minus = oracle.e4m3_encode(np.array([64.0, 128.0, -128.0]))
    cache.ks[:] = 2.0 ** -6
    for b, (first, second) in enumerate([(3, 290), (127, 128)]):
        for slot in (first, second):
            cache.k[cache.table[b, slot // 64], 0, slot % 64, 0] = one
        cache.k[cache.table[b, second // 64], 0, second % 64, 1] = two
        cache.v[cache.table[b, second // 64], 0, second % 64] = minus
        cache.v[cache.table[b, first // 64], 0, first % 64] = two
    cache.vs[:] = 2.0 ** -6
    qs = K8.Queries(rng, 2, N, G, 1, 128)
    q = np.zeros((2, N, G, 128))
    q[..., 0] = 2.0 ** e * rng.uniform(5.6, 11.2, (2, N, G))          # times log2(e) / sqrt(128): 2^e * (0.7 .. 1.4)
    q[..., 1] = q[..., 0] * 2.0 ** rng.integers(-26, -17, (2, N, G))  # half a step to 256 of them
    qs.q_t, qs.q = K8.bf16(q)
    kt = np.zeros((2, N, 1, 128))
    kt[:, ::2, :, 0] = 1
    kt[:, ::2, :, 2] = 2.0 ** -20
    qs.kt_t, qs.kt = K8.bf16(kt)
    qs.vt_t, qs.vt = K8.bf16(np.full((2, N, 1, 128), 1.5))
    out, lse, status = K8.attend(K8.dev(), cache, qs)
    assert status == 0
    assert np.isfinite(lse).all() and (np.abs(out) <= 2).all()


@pytest.mark.parametrize("N", [1, 40])
def test_bad_table_entries_are_reported_as_such(N):
    """Bad entries anywhere among many requests' blocks: each time the status says so, no call takes as long as a wait
    that gives up would, and the other requests' rows are as they should be."""
    rng = np.random.default_rng(N)
    lens = [int(x) for x in rng.integers(200, 3000, 96)]
    cache = K8.Cache(rng, lens, 2, 128, 16)
    for b in range(0, len(lens), 2):
        cache.table[b, rng.integers(0, -(-lens[b] // 16))] = [-1, cache.k.shape[0], 1 << 30, -(1 << 31)][b // 2 % 4]
    qs = K8.Queries(rng, len(lens), N, 4, 2, 128)
    dev, c = K8.dev(), cache.device(K8.dev())
    args = [qs.q_t.to(dev), qs.kt_t.to(dev), qs.vt_t.to(dev), c["k_cache"], c["v_cache"], c["k_scale"], c["v_scale"],
            torch.tensor(lens, dtype=torch.int32, device=dev), torch.from_numpy(qs.n_nodes).to(dev),
            torch.from_numpy(qs.parent).to(dev), c["block_table"]]
    began, ended = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for turn in range(10):
        status = torch.zeros(1, dtype=torch.int32, device=dev)
        began.record()
        out, lse = st.tree_attention_kv8(*args, dev_status=status)
        ended.record()
        torch.cuda.synchronize()
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        assert int(status.item()) == 7
        assert not out[::2].any() and not lse[::2].any()
        assert turn == 0 or began.elapsed_time(ended) < 500  # ms (a wait gives up after a second)
    kv8_strict.check(cache, qs, out, lse, requests=[1, 33, 95])


@pytest.mark.parametrize("N,G,slots", [(3, 4, 64), (16, 1, 64), (8, 2, 64), (20, 1, 64), (63, 4, 64), (255, 3, 64), (40, 8, 10000)])
@pytest.mark.parametrize("d", [128, 64])
def test_weights_of_the_trees_keys(N, G, slots, d):
    """With no prefix the tree's keys hold all the weight, and what is rounded to bf16 is the output alone: 2^-8 of it
    (half a step), beside the weights' pair of bf16 numbers (2^-16 of each: 2^-16 A, A = sum p |v|), the exponentials
    (2^-20 A) and float32 scores and sums over at most 255 keys (2^-14 A, as derived in kv8_helpers)."""
    rng = np.random.default_rng(N + d)
    cache = K8.Cache(rng, [0, 0, 0], 1, d, 16, max_len=slots)
    qs = K8.Queries(rng, 3, N, G, 1, d, spread=0.5)
    out, lse, status = K8.attend(K8.dev(), cache, qs)
    assert status == 0
    for b in range(3):
        O = K8.exact(cache, qs, b)[0]
        mask = oracle.tree_mask(qs.parent[b], N, 0)
        x = np.where(mask[:, None], np.einsum("nhd,kd->nhk", qs.q[b], qs.kt[b, :, 0]) / np.sqrt(d), -np.inf)
        w = np.exp(x - x.max(2, keepdims=True))
        A = np.einsum("nhk,kd->nhd", w / w.sum(2, keepdims=True), np.abs(qs.vt[b, :, 0]))
        assert kv8_strict.within(out[b], O, 2.0 ** -8 * np.abs(O) + (2.0 ** -16 + 2.0 ** -20 + 2.0 ** -14) * A).all()
