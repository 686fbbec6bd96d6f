"""Key weights of packed prompts against a 64-bit form."""

import math

import pytest
import torch

import tree_speculative_decoding_split_gb300 as st
from prompt_helpers import attention, fused, key_weights, starts

pytestmark = pytest.mark.gpu


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _check(weight, q, k, lse, start, window, scale=None):
    want, off = key_weights(q, k, lse, start, window, scale)
    lo, hi = int(start[0]), int(start[-1])
    err = (weight.double() - want).abs()[:, lo:hi]
    bound = off[:, lo:hi] + 1e-37
    assert (err <= bound).all(), (err / bound).max()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 1), (8, 2), (5, 1), (6, 2), (48, 1), (128, 1), (7, 7)])
@pytest.mark.parametrize("window", [1, 37, 300])
def test_head_layouts_and_windows(d, hq, hkv, window):
    start = starts([1, 130, 0, 513, 63])
    q, k, _ = fused(_gen(hq * d), int(start[-1]), hq, hkv, d)
    _, lse, _, _ = attention(q, k, k, start)
    lse = lse.float()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    _check(st.prompt_key_weights(q, k, lse, start, window, dev_status=status), q, k, lse, start, window)
    assert int(status) == 0


@pytest.mark.parametrize("n", [1, 2, 32, 33, 127, 128, 129, 255, 256, 257, 384, 385, 511, 513, 1000])
def test_lengths(n):
    start = starts([n])
    for hq, hkv, d, window in ((4, 1, 128, 64), (2, 2, 64, 200), (8, 1, 128, 16), (1, 1, 64, 10 ** 9)):
        q, k, _ = fused(_gen(n), n, hq, hkv, d)
        lse = attention(q, k, k, start)[1].float()
        _check(st.prompt_key_weights(q, k, lse, start, window), q, k, lse, start, window)


def test_weights_of_a_whole_window_sum_to_its_rows():
    lens = [700, 40, 1]
    start = starts(lens)
    q, k, v = fused(_gen(1), 741, 8, 2, 128)
    _, lse = st.prompt_attention(q, k, v, start)
    weight = st.prompt_key_weights(q, k, lse, start, 50)
    at = start.tolist()
    for lo, hi in zip(at[:-1], at[1:]):
        rows = min(50, hi - lo) * 4
        assert ((weight[:, lo:hi].double().sum(1) - rows).abs() <= rows * 2.0 ** -14).all()


@pytest.mark.parametrize("bad", [math.inf, math.nan])
@pytest.mark.parametrize("hq,hkv", [(4, 1), (5, 1)])
def test_rows_that_do_not_count_have_no_influence(bad, hq, hkv):
    """Queries ahead of the window or of other requests, and other keys, may hold anything."""
    lens, window = [150, 400, 60], 20
    start = starts(lens, front=10)
    n = 640
    q, k, _ = fused(_gen(2), n, hq, hkv, 128)
    lse = torch.zeros((n, hq), device="cuda")
    lse[10:620] = attention(q[10:620], k[10:620], k[10:620], starts(lens))[1].float()
    want = torch.full((hkv, n), 7.0, device="cuda")
    st.prompt_key_weights(q, k, lse, start, window, weight=want)
    assert (want[:, :10] == 7).all() and (want[:, 620:] == 7).all()
    q2, k2, lse2 = q.clone(), k.clone(), lse.clone()
    for lo, hi in ((0, 140), (160, 540), (560, 600), (620, 640)):
        q2[lo:hi], lse2[lo:hi] = bad, bad
    k2[:10], k2[620:] = bad, bad
    got = torch.full((hkv, n), 7.0, device="cuda")
    st.prompt_key_weights(q2, k2, lse2, start, window, weight=got)
    assert torch.equal(got, want)
    k2 = k.clone()
    k2[200] = bad                 # one key alone
    got = st.prompt_key_weights(q, k2, lse, start, window)
    keys = torch.arange(n, device="cuda")
    keep = (keys != 200) & (keys >= 10) & (keys < 620)
    assert torch.equal(got[:, keep], want[:, keep])


def test_window_rows_with_nan_reach_the_keys_they_see():
    start = starts([300])
    q, k, _ = fused(_gen(3), 300, 4, 1, 64)
    lse = attention(q, k, k, start)[1].float()
    q = q.contiguous()
    q[290, 2] = math.nan
    weight = st.prompt_key_weights(q, k, lse, start, 32)
    assert weight[0, :291].isnan().all() and torch.isfinite(weight[0, 291:]).all()


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("row", [290, 140])
def test_window_rows_with_any_lse_reach_no_other_keys(bad, row):
    """A row whose lse is no number (its query, or a key that it sees, was none) leaves the keys behind it as they are."""
    start = starts([300])
    q, k, _ = fused(_gen(11), 300, 4, 1, 64)
    lse = attention(q, k, k, start)[1].float()
    want = st.prompt_key_weights(q, k, lse, start, 200)
    lse[row] = bad
    got = st.prompt_key_weights(q, k, lse, start, 200)
    assert torch.equal(got[0, row + 1:], want[0, row + 1:])
    seen = got[0, :row + 1]
    assert {math.inf: (seen <= want[0, :row + 1]).all(), -math.inf: (seen == math.inf).all()}.get(bad, seen.isnan().all())


def test_keys_with_infinities():
    start = starts([200])
    q, k, _ = fused(_gen(4), 200, 5, 1, 128)
    q, k = q.contiguous().abs(), k.contiguous()
    lse = torch.zeros((200, 5), device="cuda")
    k[50], k[60] = -math.inf, math.inf
    weight = st.prompt_key_weights(q, k, lse, start, 16)
    assert weight[0, 50] == 0 and weight[0, 60] == math.inf
    weight[0, 50] = weight[0, 60] = 1
    assert torch.isfinite(weight).all()


@pytest.mark.parametrize("bad", [[0, 60, 50, 100], [-1, 50, 60, 100], [0, 50, 60, 101], [5, 3], [-1, 50], [0, 101]])
def test_bad_row_start_writes_nothing(bad):
    q, k, _ = fused(_gen(5), 100, 4, 2, 128)
    weight = torch.full((2, 100), 7.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    st.prompt_key_weights(q, k, torch.zeros((100, 4), device="cuda"), torch.tensor(bad, dtype=torch.int32, device="cuda"), 8,
                          weight=weight, dev_status=status)
    assert int(status) == 7 and (weight == 7).all()


@pytest.mark.parametrize("batch", [31, 32, 33, 64])
def test_batches_with_and_without_a_list(batch):
    lens = [0 if i in (0, 7, 8, batch - 1) else 1 + (53 * i) % 400 for i in range(batch)]
    start = starts(lens)
    n = int(start[-1])
    q, k, _ = fused(_gen(batch), n, 4, 2, 64)
    lse = attention(q, k, k, start)[1].float()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    weight = st.prompt_key_weights(q, k, lse, start, 40, dev_status=status)
    _check(weight, q, k, lse, start, 40)
    bad = start.clone()
    bad[batch // 2] = -1
    weight.fill_(7)
    st.prompt_key_weights(q, k, lse, bad, 40, weight=weight, dev_status=status)
    assert int(status) == 7 and (weight == 7).all()


def test_repeated_and_captured_calls():
    n = 900
    q, k, _ = fused(_gen(6), n, 8, 2, 128)
    start = starts([300, 600])
    lse = attention(q, k, k, start)[1].float()
    want = st.prompt_key_weights(q, k, lse, start, 48)
    assert all(torch.equal(st.prompt_key_weights(q, k, lse, start, 48), want) for _ in range(3))
    weight = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        st.prompt_key_weights(q, k, lse, start, 48, weight=weight)
    weight.zero_()
    graph.replay()
    assert torch.equal(weight, want)


@pytest.mark.parametrize("hq,hkv", [(8, 1), (64, 1)])
def test_long_windows_take_several_passes(hq, hkv):
    """Windows of many chunks, stretches of odd numbers of tiles, and the same answer call after call."""
    lens = [130, 2500, 1, 129, 700, 385]
    start = starts(lens)
    q, k, _ = fused(_gen(7), int(start[-1]), hq, hkv, 64)
    lse = attention(q, k, k, start)[1].float()
    for window in (100, 333):
        weight = st.prompt_key_weights(q, k, lse, start, window)
        _check(weight, q, k, lse, start, window)
        assert all(torch.equal(st.prompt_key_weights(q, k, lse, start, window), weight) for _ in range(5))


def test_more_heads_than_shares():
    start = starts([300, 40, 129])
    q, k, _ = fused(_gen(8), 469, 100, 100, 64)
    lse = attention(q, k, k, start)[1].float()
    _check(st.prompt_key_weights(q, k, lse, start, 30), q, k, lse, start, 30)


def test_windows_past_32_bits_and_refusals():
    start = starts([10, 20])
    q, k, _ = fused(_gen(9), 30, 4, 2, 64)
    lse = torch.zeros((30, 4), device="cuda")
    assert torch.equal(st.prompt_key_weights(q, k, lse, start, 2 ** 32 + 1), st.prompt_key_weights(q, k, lse, start, 20))
    for args in ((q, k, lse.double(), start, 4), (q, k, lse[:29], start, 4), (q, k[..., :32], lse, start, 4), (q, k, lse, start.cpu(), 4)):
        with pytest.raises((TypeError, ValueError)):
            st.prompt_key_weights(*args)
    for window in (0, -1, -2 ** 40):
        with pytest.raises(st.SpecError) as e:
            st.prompt_key_weights(q, k, lse, start, window)
        assert e.value.code == 1
