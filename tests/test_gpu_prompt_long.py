"""Prompts of tens of thousands of rows, where a CTA has many items or a long stretch of keys; and prompts in a batch."""

import pytest
import torch

import tree_speculative_decoding_split_gb300 as st
from prompt_helpers import check_attention, fused, key_weights, starts

pytestmark = pytest.mark.gpu


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


@pytest.mark.parametrize("lens,hq,hkv,d", [([33001], 2, 1, 128), ([20011, 1, 300], 4, 2, 64), ([5, 17000], 5, 1, 128)])
def test_attention(lens, hq, hkv, d):
    start = starts(lens)
    q, k, v = fused(_gen(len(lens)), int(start[-1]), hq, hkv, d)
    check_attention(st.prompt_attention(q, k, v, start), q, k, v, start)


@pytest.mark.parametrize("lens,hq,hkv,d,window", [([131072], 8, 1, 128, 64), ([32768, 129, 20000], 10, 2, 64, 37), ([70001, 33], 3, 1, 128, 200)])
def test_key_weights(lens, hq, hkv, d, window):
    start = starts(lens)
    n = int(start[-1])
    q, k, _ = fused(_gen(window), n, hq, hkv, d)
    lse = torch.zeros((n, hq), device="cuda")
    for lo, hi in zip(start.tolist()[:-1], start.tolist()[1:]):  # of the windows' rows, from their scores
        w = min(window, hi - lo)
        late = torch.arange(hi - lo, device="cuda") > torch.arange(hi - lo - w, hi - lo, device="cuda")[:, None]
        for h in range(hq):
            x = q[hi - w:hi, h].double() @ k[lo:hi, h * hkv // hq].double().T / d ** 0.5
            lse[hi - w:hi, h] = torch.logsumexp(x.masked_fill_(late, -torch.inf), 1).float()
    weight = st.prompt_key_weights(q, k, lse, start, window)
    want, off = key_weights(q, k, lse, start, window)
    assert ((weight.double() - want).abs() <= off + 1e-37).all()


@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (2, 2, 64), (5, 1, 128)])
def test_attention_of_a_prompt_alone_and_in_a_batch(hq, hkv, d):
    """To the bit, wherever it lies."""
    gen, n = _gen(hq), 700
    q, k, v = fused(gen, n, hq, hkv, d)
    want = st.prompt_attention(q, k, v, starts([n]))
    others = [300, 1, 0, 129, 64]
    for ahead in range(len(others) + 1):
        start = starts(others[:ahead] + [n] + others[ahead:])
        at, total = int(start[ahead]), int(start[-1])
        q2, k2, v2 = (x.clone() for x in fused(gen, total, hq, hkv, d))
        q2[at:at + n], k2[at:at + n], v2[at:at + n] = q, k, v
        got = st.prompt_attention(q2, k2, v2, start)
        assert all(torch.equal(a[at:at + n], b) for a, b in zip(got, want))
