"""A row of the prompt attention is its own, to the bit, whatever the rows beside it see."""

import math

import pytest
import torch

import tree_speculative_decoding_split_gb300 as st
from prompt_helpers import fused, starts

pytestmark = pytest.mark.gpu


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _same(got, want, keep):
    for x, y in zip(got, want):
        assert torch.equal(x[keep], y[keep])


@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (2, 2, 64), (5, 1, 128), (4, 4, 128)])
@pytest.mark.parametrize("kind", ["channel", "large", "sign"])
def test_unseen_keys_have_no_influence_on_rows_beside(hq, hkv, d, kind):
    """Keys with an infinity in one channel, or so large that rows that see them move their reference, beside rows that
    do not see them."""
    start = starts([150, 700, 60])
    rows = torch.arange(910, device="cuda")
    q, k, v = fused(_gen(hq * d), 910, hq, hkv, d)
    clean = [x.clone() for x in st.prompt_attention(q, k, v, start)]
    for at in (3, 101, 149, 150, 171, 277, 278, 313, 449, 555, 849, 909):
        k2 = k.clone()
        if kind == "channel":
            k2[at, :, 5] = math.inf
        elif kind == "large":
            k2[at] = k2[at] * 2.0 ** 20
        else:
            k2[at] = q[at, ::hq // hkv].sign() * 60.0
        end = next(e for e in start.tolist()[1:] if e > at)
        _same(st.prompt_attention(q, k2, v, start), clean, (rows < at) | (rows >= end))


@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (2, 2, 64), (5, 1, 128)])
@pytest.mark.parametrize("times", [2.0 ** 6, 2.0 ** 20])
def test_queries_of_others_have_no_influence(hq, hkv, d, times):
    """A request's last rows lie beside the next one's first, and those of no request, in a group."""
    start = starts([150, 300, 60], front=5)
    n = 540
    q, k, v = fused(_gen(hq + d), n, hq, hkv, d)
    clean = [x.clone() for x in st.prompt_attention(q, k, v, start)]
    for lo, hi in ((0, 5), (155, 170), (455, 460), (515, 540)):
        q2 = q.clone()
        q2[lo:hi] = q2[lo:hi] * times
        got = st.prompt_attention(q2, k, v, start)
        rows = torch.arange(n, device="cuda")
        _same(got, clean, (rows >= 5) & (rows < 515) & ((rows < lo) | (rows >= hi)))


@pytest.mark.parametrize("beside", [0, 1, 40])
def test_heads_have_no_influence_on_each_other(beside):
    """Heads of one group share its warps: one whose scores grow from tile to tile leaves the others' bits."""
    n, start = 640, starts([640])
    q, k, v = fused(_gen(9 + beside), n, 8, 1, 128)
    clean = [x.clone() for x in st.prompt_attention(q, k, v, start)]
    q2 = q.clone()
    q2[:, 3] = q2[:, 3] * (1 + beside * torch.arange(n, device="cuda")[:, None] / 16.0)
    q2[:, 3, 0] = 4.0 + beside
    got = st.prompt_attention(q2, k, v, start)
    others = [0, 1, 2, 4, 5, 6, 7]
    assert torch.equal(got[0][:, others], clean[0][:, others]) and torch.equal(got[1][:, others], clean[1][:, others])
