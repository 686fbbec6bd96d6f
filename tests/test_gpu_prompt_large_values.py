"""Prompt attention with V near the ends of float32, and scores that grow."""

import math

import pytest
import torch

import tree_speculative_decoding_split_gb300 as st
from prompt_helpers import EPS, attention, check_attention, fused, score_error, starts

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


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("power", [-100, -118, -126, -130])
def test_small_values(d, power):
    """V down to bf16's smallest numbers.  Beside the bound of ordinary ones: half a step of bf16's smallest numbers (2^-134),
    and a step of float32's (2^-149) for each of n sums, of weights 2^-12 times their own."""
    n, start = 300, starts([300])
    q, k, v = fused(_gen(-power), n, 4, 2, d)
    v = (v.float() * 2.0 ** power).bfloat16()
    out, _ = st.prompt_attention(q, k, v, start)
    want, _, mag, size = attention(q, k, v, start)
    err = score_error(size, 1 / math.sqrt(d), d)[..., None]
    bound = (1 + EPS) * mag * (EPS + 2 * err + (n + 8) * 2.0 ** -23) + EPS * want.abs() + 2.0 ** -134 + n * 2.0 ** -137
    assert ((out.double() - want).abs() <= bound).all()


@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (2, 2, 64)])
@pytest.mark.parametrize("rise", [5.0, 10.0, 40.0, 200.0])
def test_scores_that_rise_along_the_prompt(hq, hkv, d, rise):
    """Rows whose reference moves now and then, each at its own tile."""
    n, start = 1500, starts([1500])
    q, k, v = (x.clone() for x in fused(_gen(int(rise)), n, hq, hkv, d))
    q[..., 0] = 8.0
    k[..., 0] = (torch.arange(n, device="cuda") / n * rise * math.sqrt(d) / 8.0)[:, None].bfloat16()
    check_attention(st.prompt_attention(q, k, v, start), q, k, v, start)


@pytest.mark.parametrize("scale", [1e-38, 1e-31, 1e-29, 1e-10])
def test_small_scales(scale):
    """A reference above the maximum in the scores' units, which are large where the scale is small."""
    start = starts([300, 1, 130])
    q, k, v = fused(_gen(3), 431, 4, 2, 64)
    check_attention(st.prompt_attention(q, k, v, start, scale=scale), q, k, v, start, scale)
    big = (q.float() * 2.0 ** 60).bfloat16()  # scores of up to 1e20
    check_attention(st.prompt_attention(big, k, v, start, scale=scale), big, k, v, start, scale)
