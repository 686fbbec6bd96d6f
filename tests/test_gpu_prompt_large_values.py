"""Prompt attention with V near the ends of float32."""

import math

import pytest
import torch

import tree_speculative_decoding_split_gb300 as st
from prompt_helpers import check_attention, starts

pytestmark = pytest.mark.gpu


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("octaves", [5.0, 7.75, 9.0, 14.875, 15.5, 30.0])
def test_large_values_behind_grown_scores(d, octaves):
    """One later key stands above the rows' first tile: weights of up to 2^8 times V lie within float32, so do outputs.
    |V| is below 2^119, and a row's weights, all but one key's being 1 at most, sum up to less than 2^9."""
    n, start = 400, starts([400])
    q = torch.zeros((n, 2, d), device="cuda")
    q[..., 0] = 1.0
    k = torch.zeros((n, 1, d), device="cuda")
    k[200, 0, 0] = octaves * math.log(2)
    gen = _gen(int(octaves * 8))
    v = (torch.rand((n, 1, d), generator=gen, device="cuda") * 2 - 1) * 2.0 ** 118
    q, k, v = q.bfloat16(), k.bfloat16(), v.bfloat16()
    got = st.prompt_attention(q, k, v, start, scale=1.0)
    assert torch.isfinite(got[0]).all()
    check_attention(got, q, k, v, start, 1.0)
