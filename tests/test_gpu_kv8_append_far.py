"""Appending to a request whose table has room for more slots than a 32-bit length can count."""

import numpy as np
import pytest
import torch

import oracle
import tree_speculative_decoding_split_gb300 as st
import kv8_helpers as K8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("form", ["rows", "path"])
@pytest.mark.parametrize("add,served", [(3, True), (4, True), (5, False), (40, False)])
def test_lengths_end_at_the_largest_number(form, add, served):
    dev = K8.dev()
    rng = np.random.default_rng(add)
    start, bs = 2 ** 31 - 5, 256
    table = torch.full((2, 2 ** 23 + 1), -1, dtype=torch.int32, device=dev)
    table[0, -2:] = torch.tensor([2, 1], dtype=torch.int32, device=dev)
    table[1, 0] = 0
    codes = torch.zeros((3, 1, bs, 64), dtype=torch.uint8, device=dev)
    pools = [codes.clone().view(torch.float8_e4m3fn) for _ in range(2)]
    scales = [torch.ones((3, 1), device=dev) for _ in range(2)]
    seq = torch.tensor([start, 0], dtype=torch.int32, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    rows_t, rows = K8.bf16(rng.standard_normal((2, add, 1, 64)) * 1000)
    kw = dict(dev_status=status)
    x = rows_t.to(dev)
    if form == "rows":
        x = x.reshape(2 * add, 1, 64)
        kw["row_start"] = torch.tensor([0, add, 2 * add], dtype=torch.int32, device=dev)
    else:
        kw["path"] = torch.arange(add, dtype=torch.int32, device=dev).repeat(2, 1)
        kw["accept_len"] = torch.full((2,), add - 1, dtype=torch.int32, device=dev)
    new_len = st.kv8_append(x, x.clone(), *pools, *scales, seq, table, **kw)
    torch.cuda.synchronize()
    assert int(status.item()) == (0 if served else 7)
    assert new_len.tolist() == [start + add if served else start, add]
    want, want_scale = np.zeros((3, 1, bs, 64), np.uint8), np.ones((3, 1))
    oracle.append_rows(rows[1], want, want_scale, 0, [0], bs)
    if served:
        oracle.append_rows(rows[0], want, want_scale, bs - 5, [2, 1], bs)
    for c in range(2):
        assert np.array_equal(pools[c].view(torch.uint8).cpu().numpy(), want)
        assert np.array_equal(scales[c].cpu().numpy(), want_scale.astype(np.float32))
