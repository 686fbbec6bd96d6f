"""Rows whose offsets pass 32 bits: a few rows, each far from the next."""

import pytest
import torch

import tree_speculative_decoding_split_gb300 as st
from prompt_helpers import check_attention, kept, key_weights, rows, starts

pytestmark = pytest.mark.gpu

STEP = 1 << 22  # elements between rows: 700 rows are 2.9e9 elements


@pytest.fixture(scope="module")
def far():
    """q, k and v as views of rows STEP elements apart, and the same rows side by side."""
    n, hq, hkv, d = 700, 8, 2, 64
    base = torch.empty(n * STEP, dtype=torch.bfloat16, device="cuda")
    near = rows(torch.Generator(device="cuda").manual_seed(1), n, hq + 2 * hkv, d)
    wide = torch.as_strided(base, (n, hq + 2 * hkv, d), (STEP, d, 1))
    wide.copy_(near)
    split = lambda x: (x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:])
    yield split(wide), split(near)
    del base, wide


def test_far_rows_as_near_ones(far):
    (q, k, v), (q2, k2, v2) = far
    start = starts([300, 400])
    got = st.prompt_attention(q, k, v, start)
    check_attention(got, q2, k2, v2, start)
    weight = st.prompt_key_weights(q, k, got[1], start, 20)
    want, off = key_weights(q2, k2, got[1], start, 20)
    assert ((weight.double() - want).abs() <= off + 1e-37).all()
    k_out, v_out, index, keep_start, _ = st.kv_keep(k, v, weight, start, 50, 2, 5)
    chosen = kept(weight.cpu(), start.cpu(), 50, 2, 5)
    assert index.tolist() == [list(x) for h in chosen for x in zip(*h)] and keep_start.tolist() == [0, 50, 100]
    at = index.long() + torch.tensor([0] * 50 + [300] * 50, device="cuda")[:, None]
    head = torch.arange(2, device="cuda")
    assert torch.equal(k_out, k2[at, head]) and torch.equal(v_out, v2[at, head])


def test_far_rows_turn_in_place(far):
    (q, k, _), (q2, k2, _) = far
    pos = torch.arange(700, device="cuda", dtype=torch.int32)
    turns = st.rope_table(64).cuda()
    want = st.rope(q2, k2, pos, turns)
    st.rope(q, k, pos, turns, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
