"""rows_out of kv_keep beside a caller's own outputs."""

import pytest
import torch

import tree_speculative_decoding_split_gb300 as st
from prompt_helpers import rows, starts

pytestmark = pytest.mark.gpu


def _outputs(n_out, batch):
    i32 = dict(dtype=torch.int32, device="cuda")
    return (torch.zeros((n_out, 2, 64), dtype=torch.bfloat16, device="cuda"), torch.zeros((n_out, 2, 64), dtype=torch.bfloat16, device="cuda"),
            torch.zeros((n_out, 2), **i32), torch.zeros(batch + 1, **i32), torch.zeros(batch, **i32))


def test_a_bound_other_than_the_outputs_rows_is_refused():
    gen = torch.Generator(device="cuda").manual_seed(1)
    k = rows(gen, 60, 2, 64)
    w = torch.rand((2, 60), generator=gen, device="cuda")
    start = starts([25, 35])
    for bound in (10, 39, 41):
        with pytest.raises(ValueError):
            st.kv_keep(k, k, w, start, 20, rows_out=bound, outputs=_outputs(40, 2))
    got = st.kv_keep(k, k, w, start, 20, rows_out=40, outputs=_outputs(40, 2))
    want = st.kv_keep(k, k, w, start, 20)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
