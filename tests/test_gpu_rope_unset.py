"""Positions that no request gives: rows in front of, behind and, where row_start is refused, inside the requests."""

import pytest
import torch

import tree_speculative_decoding_split_gb300 as st
from prompt_helpers import rows, starts

pytestmark = pytest.mark.gpu


def _dirty(n):
    """Leaves a freed block of n numbers behind that look like positions."""
    x = torch.full((n,), 12345, dtype=torch.int32, device="cuda")
    del x


@pytest.mark.parametrize("stream", [False, True])
@pytest.mark.parametrize("lens,front,behind", [([5, 0, 9], 3, 8), ([0], 4, 3), ([2000, 1], 1030, 2000)])
def test_rows_of_no_request_have_no_position(lens, front, behind, stream):
    start = starts(lens, front=front)
    n = int(start[-1]) + behind
    pos0 = torch.arange(len(lens), device="cuda", dtype=torch.int32) * 100
    _dirty(n)
    more = dict(stream=torch.cuda.current_stream()) if stream else {}
    pos = st.rope_positions(pos0, row_start=start, n_rows=n, **more)
    want = [-1] * front + [100 * b + j for b, m in enumerate(lens) for j in range(m)] + [-1] * behind
    assert pos.tolist() == want
    x = rows(torch.Generator(device="cuda").manual_seed(1), n, 3, 64)
    before = x.clone()
    q, k = x[:, :2], x[:, 2:]
    st.rope(q, k, pos, st.rope_table(64).cuda(), q_out=q, k_out=k)
    none = pos < 0
    assert torch.equal(x[none], before[none])


@pytest.mark.parametrize("stream", [False, True])
@pytest.mark.parametrize("bad", [[0, 60, 50, 100], [-1, 50, 60, 100], [0, 50, 60, 3001]])
def test_a_refused_row_start_gives_no_positions(bad, stream):
    n = 3000
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    _dirty(n)
    more = dict(stream=torch.cuda.current_stream()) if stream else {}
    pos = st.rope_positions(torch.zeros(3, dtype=torch.int32, device="cuda"), row_start=torch.tensor(bad, dtype=torch.int32, device="cuda"),
                            n_rows=n, dev_status=status, **more)
    assert int(status) == 7 and (pos == -1).all()


def test_a_given_buffer_keeps_what_it_holds():
    start = starts([5, 9], front=3)
    out = torch.full((30,), -7, dtype=torch.int32, device="cuda")
    pos0 = torch.zeros(2, dtype=torch.int32, device="cuda")
    st.rope_positions(pos0, row_start=start, n_rows=30, positions=out)
    assert (out[:3] == -7).all() and (out[17:] == -7).all() and out[3:17].tolist() == list(range(5)) + list(range(9))
