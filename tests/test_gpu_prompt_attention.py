"""Causal attention over packed prompts against a 64-bit form."""

import math

import pytest
import torch

import tree_speculative_decoding_split_gb300 as st
from prompt_helpers import attention, check_attention, fused, rows, starts

pytestmark = pytest.mark.gpu


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 1), (8, 2), (5, 1), (6, 2), (16, 1), (48, 1), (128, 1), (7, 7)])
def test_head_layouts(d, hq, hkv):
    start = starts([1, 130, 0, 257, 63])
    q, k, v = fused(_gen(hq * d), int(start[-1]), hq, hkv, d)
    status = _status()
    got = st.prompt_attention(q, k, v, start, dev_status=status)
    check_attention(got, q, k, v, start)
    assert int(status) == 0


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 383, 384, 385, 511, 513, 1000])
def test_lengths(n):
    start = starts([n])
    for hq, hkv, d in ((4, 1, 128), (2, 2, 64), (1, 1, 128)):
        q, k, v = fused(_gen(n), n, hq, hkv, d)
        check_attention(st.prompt_attention(q, k, v, start), q, k, v, start)


def test_many_short_and_some_long():
    lens = [(17 * b) % 41 for b in range(300)] + [2500, 1, 700]
    start = starts(lens)
    q, k, v = fused(_gen(1), int(start[-1]), 8, 2, 128)
    check_attention(st.prompt_attention(q, k, v, start), q, k, v, start)


def test_long_prompt():
    start = starts([6001])
    q, k, v = fused(_gen(2), 6001, 8, 1, 128)
    check_attention(st.prompt_attention(q, k, v, start), q, k, v, start)


def test_rows_of_no_request_stay():
    start = starts([40, 0, 100], front=30)
    n = 200
    q, k, v = fused(_gen(3), n, 4, 2, 64)
    for x in (q, k, v):
        x[:30] = math.nan
        x[170:] = math.inf
    out = torch.full((n, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((n, 4), 7.0, device="cuda")
    st.prompt_attention(q, k, v, start, out=out, lse=lse)
    for x in (out, lse):
        assert (x[:30] == 7).all() and (x[170:] == 7).all()
    check_attention((out[30:170], lse[30:170]), q[30:170], k[30:170], v[30:170], starts([40, 0, 100]))


@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (2, 2, 64), (5, 1, 128)])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_unseen_keys_have_no_influence(hq, hkv, d, bad):
    """Rows before a key with infinities or NaN, and the other requests, come out to the bit as without it."""
    lens = [150, 300, 60]
    start = starts(lens)
    q, k, v = fused(_gen(4), 510, hq, hkv, d)
    clean = st.prompt_attention(q, k, v, start)
    clean = [x.clone() for x in clean]
    for at in (0, 149, 150, 200, 277, 278, 449, 450, 509):
        k2, v2 = k.clone(), v.clone()
        k2[at], v2[at, :, ::3] = bad, bad
        got = st.prompt_attention(q, k2, v2, start)
        end = next(e for e in start.tolist()[1:] if e > at)
        for x, y in zip(got, clean):
            assert torch.equal(x[:at], y[:at]) and torch.equal(x[end:], y[end:])


@pytest.mark.parametrize("at", [0, 5, 127, 128, 200, 299])
def test_infinities_reach_the_rows_that_see_them(at):
    start = starts([300, 20])
    q, k, v = fused(_gen(5), 320, 4, 2, 128)
    v = v.contiguous()
    v[at, 0, 3], v[at, 1, 64], v[at, 1, 100] = math.inf, -math.inf, math.nan
    out, _ = st.prompt_attention(q, k, v, start)
    seen = torch.arange(320, device="cuda")
    seen = ((seen >= at) & (seen < 300))[:, None]
    assert torch.equal(out[:, :2, 3] == math.inf, seen.expand(-1, 2))
    assert torch.equal(out[:, 2:, 64] == -math.inf, seen.expand(-1, 2))
    assert torch.equal(out[:, 2:, 100].isnan(), seen.expand(-1, 2))
    rest = torch.isfinite(out)
    rest[:, :2, 3] = rest[:, 2:, 64] = rest[:, 2:, 100] = True
    assert rest.all()


@pytest.mark.parametrize("power", [20, 40, 60])
def test_large_scores(power):
    """Scores where one step of float32 is many units of the exponent: the largest key takes all, ties share."""
    n, d = 200, 64
    start = starts([n])
    q = torch.zeros((n, 2, d), device="cuda")
    q[..., 0] = 2.0 ** (power / 2)
    k = torch.zeros((n, 1, d), device="cuda")
    rank = torch.randperm(n, generator=torch.Generator().manual_seed(power)) // 2
    k[:, 0, 0] = (128 + rank.cuda() - n // 2) * 2.0 ** (power / 2 - 7)
    v = rows(_gen(6), n, 1, d)
    out, lse = st.prompt_attention(q.bfloat16(), k.bfloat16(), v, start, scale=1.0)
    assert torch.equal(k.bfloat16().float(), k)
    for i in (0, 1, 50, 127, 128, 199):
        top = rank[:i + 1] == rank[:i + 1].max()
        best = v[:i + 1, 0][top.cuda()].double()
        err = (out[i, 0].double() - best.mean(0)).abs()
        assert (err <= 2 * 2.0 ** -8 * best.abs().mean(0) + 1e-30).all()
        want = 2.0 ** (power / 2) * float(k[:i + 1, 0, 0].max()) + math.log(int(top.sum()))  # ln of as many equal terms
        assert abs(float(lse[i, 0]) - want) <= want * 2.0 ** -22


def test_growing_scores_rescale():
    """Every tile's scores pass the ones before it, so that the running maximum moves each time."""
    n = 900
    start = starts([n])
    q, k, v = (rows(_gen(s), n, 4, 128) for s in (7, 8, 9))
    k = (k.float() * 0.1 + q[:1].float().sign() * (torch.arange(n, device="cuda") / 60.0)[:, None, None]).bfloat16()
    q = (q.float().abs() * q[:1].float().sign()).bfloat16()
    check_attention(st.prompt_attention(q, k, v, start), q, k, v, start)


def test_strides_scale_and_workspace():
    start = starts([100, 101])
    x = rows(_gen(10), 201, 40, 64)
    q, k, v = x[:, 3:11], x[:, 20:24], x[:, 30:34]
    ws = torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    got = st.prompt_attention(q, k, v, start, scale=0.3, workspace=ws)
    check_attention(got, q, k, v, start, 0.3)
    whole = st.prompt_attention(q.contiguous(), k.contiguous(), v.contiguous(), start, scale=0.3)
    assert all(torch.equal(a, b) for a, b in zip(got, whole))
    with pytest.raises(ValueError):
        st.prompt_attention(q, k, v, start, workspace=ws[:16])


@pytest.mark.parametrize("bad", [[0, 60, 50, 100], [-1, 50, 60, 100], [0, 50, 60, 101], [5, 3], [-1, 50], [0, 101]])
def test_bad_row_start_writes_nothing(bad):
    q, k, v = fused(_gen(11), 100, 4, 2, 128)
    out, lse = torch.full((100, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((100, 4), 7.0, device="cuda")
    status = _status()
    st.prompt_attention(q, k, v, torch.tensor(bad, dtype=torch.int32, device="cuda"), out=out, lse=lse, dev_status=status)
    assert int(status) == 7 and (out == 7).all() and (lse == 7).all()


@pytest.mark.parametrize("batch", [31, 32, 33, 64])
@pytest.mark.parametrize("heads", [1, 40])
def test_batches_with_and_without_a_list(batch, heads):
    """Pieces found in row_start by the kernel or listed ahead of it, in order or by work; requests without rows at the ends."""
    lens = [0 if i in (0, 7, 8, batch - 1) else 1 + (53 * i) % 140 for i in range(batch)]
    start = starts(lens)
    n = int(start[-1])
    q, k, v = fused(_gen(batch), n, heads, heads, 64)
    status = _status()
    out, lse = st.prompt_attention(q, k, v, start, dev_status=status)
    check_attention((out, lse), q, k, v, start)
    bad = start.clone()
    bad[batch // 2] = n + 1
    out.fill_(7)
    st.prompt_attention(q, k, v, bad, out=out, lse=lse, dev_status=status)
    assert int(status) == 7 and (out == 7).all()


def test_no_rows():
    start = starts([0, 0])
    q = torch.empty((0, 4, 128), dtype=torch.bfloat16, device="cuda")
    status = _status()
    out, lse = st.prompt_attention(q, q[:, :2], q[:, :2], start, dev_status=status)
    assert out.shape == (0, 4, 128) and lse.shape == (0, 4) and int(status) == 0


def test_calls_repeat_and_streams_do_not_meet():
    start = starts([700, 20, 333])
    q, k, v = fused(_gen(12), 1053, 16, 4, 128)
    want = [x.clone() for x in st.prompt_attention(q, k, v, start)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got += [st.prompt_attention(q, k, v, start) for _ in range(3)]
    torch.cuda.synchronize()
    for out, lse in got:
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("all_lens", [([100, 500], [599, 1], [0, 600], [300, 300]), ([600], [1], [0], [300])])
def test_captured_calls_follow_lengths_on_the_device(all_lens):
    n = 600
    q, k, v = fused(_gen(13), n, 8, 2, 64)
    start = starts(all_lens[0])
    out, lse = torch.empty((n, 8, 64), dtype=torch.bfloat16, device="cuda"), torch.empty((n, 8), device="cuda")
    ws = torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    st.prompt_attention(q, k, v, start, out=out, lse=lse, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        st.prompt_attention(q, k, v, start, out=out, lse=lse, workspace=ws)
        st.prompt_attention(q, k, v, start, out=out, lse=lse, workspace=ws)
    for lens in all_lens:
        start.copy_(starts(lens))
        graph.replay()
        check_attention((out, lse), q, k, v, start)


def test_a_first_tile_of_infinities():
    """Rows whose first 128 scores are all -inf (K rows of -inf) take their weights from what follows, however small."""
    n, d = 300, 64
    start = starts([n])
    q = torch.ones((n, 2, d), device="cuda").bfloat16()
    k = torch.full((n, 1, d), -4.0, device="cuda")
    k[:128, 0, 0] = -math.inf
    k[128:, 0, 1] = torch.arange(n - 128, device="cuda") % 8 * 0.5
    v = rows(_gen(14), n, 1, d)
    out, lse = st.prompt_attention(q, k.bfloat16(), v, start, scale=1.0)
    want, want_lse, mag, _ = attention(q[128:], k[128:].bfloat16(), v[128:], starts([n - 128]), 1.0)
    assert ((out[128:].double() - want).abs() <= 2.1 * 2.0 ** -8 * mag + 1e-30).all()
    assert ((lse[128:].double() - want_lse).abs() <= 2.0 ** -20 * want_lse.abs()).all()


def test_many_heads_and_unaligned_rows():
    """More heads than SMs, and outputs that begin 16 bytes off a 32-byte sector."""
    start = starts([70, 200])
    q, k, v = fused(_gen(15), 270, 200, 200, 64)
    out = torch.zeros(270 * 200 * 64 + 8, dtype=torch.bfloat16, device="cuda")[8:].view(270, 200, 64)
    assert out.data_ptr() % 32 == 16
    got = st.prompt_attention(q, k, v, start, out=out)
    check_attention(got, q, k, v, start)


def test_refusals():
    start = starts([10, 20])
    q, k, v = fused(_gen(16), 30, 4, 2, 64)
    for args in ((q.float(), k, v, start), (q, k.half(), v, start), (q, k, v, start.long()), (q, k, v, start.cpu()), (q.cpu(), k, v, start),
                 (q, k[:29], v, start), (q, k, v[:, :1], start), (q, k, v[..., :32], start), (q[None], k, v, start),
                 (q.transpose(0, 1), k, v, start), (q[..., ::2], k[..., ::2], v[..., ::2], start), (q, k, v[::2], start)):
        with pytest.raises((TypeError, ValueError)):
            st.prompt_attention(*args)
    for args, code in (((q.float(), k.float(), v.float(), start), 2), ((q[:, :3], k, v, start), 1),
                       ((q[..., :32], k[..., :32], v[..., :32], start), 2), ((q.reshape(-1)[4:4 + 29 * 256].view(29, 4, 64), k[:29], v[:29], start), 1)):
        q2 = args[0]
        if q2.shape[2] == 32:
            args = tuple(x.contiguous() for x in args[:3]) + args[3:]
        with pytest.raises(st.SpecError) as e:
            st.prompt_attention(*args)
        assert e.value.code == code
    out = torch.empty((30, 4, 64), dtype=torch.bfloat16, device="cuda")
    for more in (dict(out=out[:29]), dict(out=out.float()), dict(lse=torch.empty((30, 2), device="cuda")), dict(dev_status=start.long())):
        with pytest.raises((TypeError, ValueError)):
            st.prompt_attention(q, k, v, start, **more)
