"""lse of prompt attention for rows of few keys, where it may lie near 0."""

import math

import pytest
import torch

import tree_speculative_decoding_split_gb300 as st
from prompt_helpers import attention, fused, score_error, starts

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,scale", [(64, 0.0), (128, 0.0), (128, 0.37), (64, 1e-3)])
@pytest.mark.parametrize("spread", [0.01, 0.3, 1.0])
def test_lse_of_few_keys(d, scale, spread):
    """Beside the score's own error: an exponential of a number of 16 at most (2^-21 of rounding, 2^-22 of itself), up to
    four terms (2^-22), a logarithm (2^-23 of itself at most, as is the sum it is part of): 2^-20, and 2^-22 of lse."""
    lens = [1, 2, 3, 4] * 100
    start = starts(lens)
    q, k, v = fused(torch.Generator(device="cuda").manual_seed(d), int(start[-1]), 4, 2, d)
    q = (q.float() * spread).bfloat16()
    _, lse = st.prompt_attention(q, k, v, start, scale=scale)
    scale = scale or 1 / math.sqrt(d)
    _, want, _, size = attention(q, k, v, start, scale)
    bound = score_error(size, scale, d) + 2.0 ** -20 + want.abs() * 2.0 ** -22
    assert ((lse.double() - want).abs() <= bound).all(), ((lse.double() - want).abs() / bound).max()
