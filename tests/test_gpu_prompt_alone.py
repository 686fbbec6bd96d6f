"""Key weights of a prompt do not depend on the batch that it comes in, to the bit."""

import pytest
import torch

import tree_speculative_decoding_split_gb300 as st
from prompt_helpers import fused, starts

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq,hkv,d,window", [(8, 1, 128, 48), (8, 2, 64, 90), (5, 1, 128, 70), (16, 2, 128, 300), (4, 4, 64, 200)])
@pytest.mark.parametrize("batch", [3, 40])
def test_weights_alone_and_in_a_batch(hq, hkv, d, window, batch):
    """The same prompt by itself, and behind and ahead of others of odd and even numbers of tiles."""
    gen = torch.Generator(device="cuda").manual_seed(hq + window)
    others = [700, 129, 1, 0, 260] + [(37 * i) % 300 for i in range(batch - 3)]
    n = 1500
    q, k, v = fused(gen, n, hq, hkv, d)
    _, lse = st.prompt_attention(q, k, v, starts([n]))
    want = st.prompt_key_weights(q, k, lse, starts([n]), window)
    for ahead in range(0, len(others), 2 if batch < 10 else 9):
        lens = others[:ahead] + [n] + others[ahead:]
        start = starts(lens)
        at = int(start[ahead])
        total = int(start[-1])
        q2, k2, _ = fused(gen, total, hq, hkv, d)
        lse2 = torch.zeros((total, hq), device="cuda")
        q2, k2 = q2.clone(), k2.clone()
        q2[at:at + n], k2[at:at + n], lse2[at:at + n] = q, k, lse
        got = st.prompt_key_weights(q2, k2, lse2, start, window)
        assert torch.equal(got[:, at:at + n], want)
