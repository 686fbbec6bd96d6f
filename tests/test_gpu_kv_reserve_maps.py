"""Slot maps of no entries: a bound of 0 rows is a bound, on both ways of marshalling."""

import pytest
import torch

import tree_speculative_decoding_split_gb300 as st
import kv8_helpers as K8

pytestmark = pytest.mark.gpu


def _state(B):
    i = lambda x: torch.tensor(x, dtype=torch.int32, device=K8.dev())  # noqa: E731
    table = torch.full((B, 8), -1, dtype=torch.int32, device=K8.dev())
    table[:, :2] = torch.arange(2 * B, device=K8.dev()).view(B, 2)
    return dict(block_table=table, n_blocks=i([2] * B), free_list=torch.arange(8 * B, dtype=torch.int32, device=K8.dev()).flip(0),
                free_count=i([6 * B]))


@pytest.mark.parametrize("B", [2, 90])
@pytest.mark.parametrize("kind", ["slot_cap", "slot_map"])
@pytest.mark.parametrize("native", [True, False])
def test_a_map_without_entries_allows_no_row(B, kind, native):
    dev = K8.dev()
    kw = dict(slot_cap=0) if kind == "slot_cap" else dict(slot_map=torch.empty(0, dtype=torch.int64, device=dev))
    if not native:
        kw["stream"] = torch.cuda.current_stream()
    lens = torch.full((B,), 20, dtype=torch.int32, device=dev)
    new = torch.zeros(B, dtype=torch.int32, device=dev)
    new[B - 1] = 20
    s, status = _state(B), torch.zeros(1, dtype=torch.int32, device=dev)
    before = {k: v.clone() for k, v in s.items()}
    slots, starts = st.kv_reserve(lens, new, block_size=16, dev_status=status, **s, **kw)
    torch.cuda.synchronize()
    assert int(status.item()) == 7 and slots.numel() == 0 and not starts.any()
    for k in s:
        assert torch.equal(s[k], before[k]), k
    # no new rows: served, and what is not needed goes back
    lens[0] = 3
    new.zero_()
    status.zero_()
    slots, starts = st.kv_reserve(lens, new, block_size=16, dev_status=status, **s, **kw)
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and slots.numel() == 0 and not starts.any()
    assert s["n_blocks"].tolist() == [1] + [2] * (B - 1) and int(s["free_count"].item()) == 6 * B + 1
