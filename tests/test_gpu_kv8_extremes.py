"""Tree attention over the 8-bit cache at the ends of what its inputs may hold: rows of zeros, rows next to bf16's
smallest and largest numbers."""

import numpy as np
import pytest

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
