"""Rows kept for a budget against a sort on the host."""

import math

import pytest
import torch

import tree_speculative_decoding_split_gb300 as st
from prompt_helpers import kept, rows, starts

pytestmark = pytest.mark.gpu


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _run(k, v, weight, start, budget, first=0, last=0, **more):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    k_out, v_out, index, keep_start, n_keep = st.kv_keep(k, v, weight, start, budget, first=first, last=last, dev_status=status,
                                                         **more)
    want = kept(weight.cpu(), start.cpu(), budget, first, last)
    counts = [len(h[0]) for h in want]
    assert n_keep.tolist() == counts
    assert keep_start.tolist() == [sum(counts[:b]) for b in range(len(counts) + 1)]
    flat = [list(r) for h in want for r in zip(*h)]
    total = sum(counts)
    assert index[:total].tolist() == flat
    at = torch.tensor(flat, device="cuda").reshape(total, weight.shape[0])
    base = torch.repeat_interleave(start[:-1].long(), torch.tensor(counts, device="cuda"))
    source, head = base[:, None] + at, torch.arange(weight.shape[0], device="cuda")
    assert torch.equal(k_out[:total], k[source, head]) and torch.equal(v_out[:total], v[source, head])
    assert int(status) == 0


def _weights(gen, heads, n):
    w = torch.randn((heads, n), generator=gen, device="cuda").exp()
    return torch.where(torch.rand((heads, n), generator=gen, device="cuda") < 0.2, torch.zeros_like(w), w)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,budget,first,last", [([1], 1, 0, 0), ([2], 1, 0, 1), ([10, 0, 5, 100], 7, 2, 3), ([100, 99], 100, 4, 8),
                                                    ([101, 500], 100, 50, 50), ([33, 1025, 31], 32, 0, 0), ([4097, 2048], 1000, 4, 64)])
def test_budgets(dtype, d, lens, budget, first, last):
    start = starts(lens)
    n = int(start[-1])
    gen = _gen(n)
    x = rows(gen, n, 7, d, dtype)
    _run(x[:, :3], x[:, 3:6], _weights(gen, 3, n), start, budget, first, last)


@pytest.mark.parametrize("heads", [1, 2, 8, 40])
def test_long_prompts(heads):
    """One request with clusters of eight CTAs down to single ones; stretches longer than a CTA holds."""
    n = 100003 if heads > 2 else 400000
    start = starts([n])
    gen = _gen(heads)
    k = torch.arange(n, device="cuda").float()[:, None, None].expand(n, heads, 64).contiguous().bfloat16()
    _run(k, k, _weights(gen, heads, n), start, 777, 3, 5)


def test_more_rows_than_a_single_cta_holds():
    """So many heads that no CTA has another beside it, and more rows than shared memory keeps."""
    heads, n = 80, 42000
    gen = _gen(5)
    k = torch.arange(n, device="cuda").float()[:, None, None].expand(n, heads, 64).contiguous().bfloat16()
    _run(k, k, _weights(gen, heads, n), starts([n]), 600, 1, 2)
    w = torch.zeros((heads, n), device="cuda")
    w[::2, 41000:41500] = 1  # what stays lies behind what is held; elsewhere all is equal
    _run(k, k, w, starts([n]), 600)


@pytest.mark.parametrize("batch", [31, 32, 33, 70])
def test_batches_counted_by_warps_and_by_blocks(batch):
    gen = _gen(batch)
    lens = [(37 * i) % 90 for i in range(batch)]
    start = starts(lens)
    n = int(start[-1])
    x = rows(gen, n, 2, 64)
    _run(x, x, _weights(gen, 2, n), start, 40, 2, 3)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kept_rows = sum(min(c, 40) for c in lens)
    out = st.kv_keep(x, x, _weights(gen, 2, n), start, 40, rows_out=kept_rows - 1, dev_status=status)
    assert int(status) == 7 and not out[3].any() and not out[4].any()


@pytest.mark.parametrize("kind", ["equal", "zeros", "two", "negative", "special", "steps"])
def test_ties_and_order(kind):
    n, gen = 5000, _gen(11)
    w = {"equal": torch.ones((2, n), device="cuda"), "zeros": torch.zeros((2, n), device="cuda"),
         "two": (torch.arange(2 * n, device="cuda") % 7 == 0).float().view(2, n), "negative": -_weights(gen, 2, n),
         "special": _weights(gen, 2, n), "steps": 1 + torch.randint(0, 900, (2, n), generator=gen, device="cuda") * 2.0 ** -23}[kind]
    if kind == "zeros":
        w[:, ::2] = -0.0
    if kind == "special":
        w[0, ::5], w[0, 1::5], w[1, ::3], w[1, 1::3] = math.nan, math.inf, -math.inf, math.nan
    k = rows(gen, n, 2, 64)
    for budget in (1, 64, 999, 2500, 4999):
        _run(k, k, w, starts([n]), budget)
        if budget > 20:
            _run(k, k, w, starts([n]), budget, 10, 10)


def test_rows_of_no_request_and_behind_the_kept_ones_stay():
    start = starts([50, 0, 20], front=7)
    gen = _gen(12)
    k, v, w = rows(gen, 90, 2, 64), rows(gen, 90, 2, 64), _weights(gen, 2, 90)
    w[:, :7] = w[:, 77:] = math.inf
    outputs = (torch.full((60, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((60, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda"),
               torch.full((60, 2), -7, dtype=torch.int32, device="cuda"), torch.empty(4, dtype=torch.int32, device="cuda"),
               torch.empty(3, dtype=torch.int32, device="cuda"))
    _run(k, v, w, start, 30, 1, 1, outputs=outputs)
    assert all((x[50:] == (-7 if x.dtype == torch.int32 else 7)).all() for x in outputs[:3])


@pytest.mark.parametrize("empty", [0, 2000])
def test_refusals_on_the_device(empty):
    """Among few requests and (with empty ones behind) among many."""
    k = rows(_gen(13), 100, 2, 64)
    w = _weights(_gen(14), 2, 100)
    for start, rows_out in (([0, 60, 50, 100], 100), ([-1, 50, 60, 100], 100), ([0, 50, 60, 101], 100), ([0, 50, 60, 100], 49)):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        start = start + [start[-1]] * empty
        outputs = (torch.full((rows_out, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda"),
                   torch.full((rows_out, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda"),
                   torch.full((rows_out, 2), -7, dtype=torch.int32, device="cuda"),
                   torch.full((len(start),), -7, dtype=torch.int32, device="cuda"),
                   torch.full((len(start) - 1,), -7, dtype=torch.int32, device="cuda"))
        st.kv_keep(k, k, w, torch.tensor(start, dtype=torch.int32, device="cuda"), 20, outputs=outputs, dev_status=status)
        assert int(status) == 7 and (outputs[0] == 7).all() and (outputs[1] == 7).all() and (outputs[2] == -7).all()
        assert not outputs[3].any() and not outputs[4].any()


@pytest.mark.parametrize("batch", [700, 1024, 1025, 3000])
def test_many_requests(batch):
    lens = [(31 * b) % 97 for b in range(batch)]
    start = starts(lens)
    n = int(start[-1])
    gen = _gen(15)
    _run(rows(gen, n, 3, 64), rows(gen, n, 3, 64), _weights(gen, 3, n), start, 40, 2, 6)


def test_captured_calls_follow_lengths_on_the_device():
    gen = _gen(16)
    k, w = rows(gen, 3000, 2, 128), _weights(gen, 2, 3000)
    start = starts([1000, 2000])
    eager = st.kv_keep(k, k, w, start, 300, rows_out=600)
    outputs = tuple(torch.empty_like(x) for x in eager)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        st.kv_keep(k, k, w, start, 300, outputs=outputs)
    for lens in ([1000, 2000], [1, 2999], [0, 3000], [299, 2701]):
        start.copy_(starts(lens))
        graph.replay()
        want = st.kv_keep(k, k, w, start, 300, rows_out=600)
        total = int(want[3][-1])
        assert all(torch.equal(a[:total], b[:total]) for a, b in zip(outputs[:3], want[:3]))
        assert torch.equal(outputs[3], want[3]) and torch.equal(outputs[4], want[4])


def test_no_rows():
    k = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.empty((2, 0), device="cuda")
    _, _, index, keep_start, n_keep = st.kv_keep(k, k, w, starts([0, 0]), 5)
    assert index.shape == (0, 2) and keep_start.tolist() == [0, 0, 0] and n_keep.tolist() == [0, 0]


def test_budgets_past_32_bits_and_refusals():
    k = rows(_gen(17), 30, 2, 64)
    w, start = _weights(_gen(18), 2, 30), starts([10, 20])
    _run(k, k, w, start, 2 ** 32 + 3)
    for args in ((k, k.float(), w, start, 4), (k, k[:29], w, start, 4), (k, k, w[:, :29], start, 4), (k, k, w.double(), start, 4),
                 (k, k, w, start.long(), 4)):
        with pytest.raises((TypeError, ValueError)):
            st.kv_keep(*args)
    for more in (dict(budget=0), dict(budget=-2 ** 33), dict(budget=4, first=3, last=2), dict(budget=4, first=-1), dict(budget=4, last=2 ** 33)):
        with pytest.raises(st.SpecError) as e:
            st.kv_keep(k, k, w, start, **more)
        assert e.value.code == 1
