"""Positions and rotation on the GPU against 64-bit forms."""

import math
import random

import pytest
import torch

import tree_speculative_decoding_split_gb300 as st
from prompt_helpers import fused, rows, starts

pytestmark = pytest.mark.gpu


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ---- positions -----------------------------------------------------------------------------------

@pytest.mark.parametrize("lens,front,behind", [([1], 0, 0), ([5, 0, 0, 3], 0, 0), ([0, 7, 0], 3, 5), ([1024, 1, 2047], 0, 1),
                                               ([3] * 2000, 2, 7), ([1] * 2048, 0, 1), ([2, 0, 1] * 700, 1, 3), ([0, 0], 4, 9)])
def test_positions_of_rows(lens, front, behind):
    start = starts(lens, front=front)
    n_rows = int(start[-1]) + behind
    pos0 = _ints([(37 * b) % 1000 for b in range(len(lens))])
    out = torch.full((n_rows,), -7, dtype=torch.int32, device="cuda")
    status = _status()
    assert st.rope_positions(pos0, row_start=start, n_rows=n_rows, positions=out, dev_status=status) is out
    want = [-7] * front + [int(p) + j for p, n in zip(pos0.tolist(), lens) for j in range(n)] + [-7] * behind
    assert out.tolist() == want and int(status) == 0


@pytest.mark.parametrize("bad", [[0, 4, 3, 8], [-1, 4, 5, 8], [0, 4, 5, 9]])
def test_bad_row_start_writes_nothing(bad):
    out = torch.full((8,), -7, dtype=torch.int32, device="cuda")
    status = _status()
    st.rope_positions(_ints([0, 0, 0]), row_start=_ints(bad), n_rows=8, positions=out, dev_status=status)
    assert int(status) == 7 and (out == -7).all()


def test_positions_past_32_bits_refuse_their_request():
    status = _status()
    top = 2 ** 31 - 1
    out = st.rope_positions(_ints([top - 1, top - 2, -1, 0]), row_start=_ints([0, 3, 6, 8, 10]), n_rows=10, dev_status=status)
    assert out.tolist() == [-1] * 3 + [top - 2, top - 1, top] + [-1] * 2 + [0, 1] and int(status) == 7


def _depth(parent, n):
    d = [0] * n
    for i in range(1, n):
        d[i] = d[parent[i]] + 1
    return d


@pytest.mark.parametrize("n_max", [1, 2, 31, 63, 255])
def test_positions_of_trees(n_max):
    rng = random.Random(n_max)
    trees, nodes = [], []
    for kind in range(6):
        n = n_max if kind < 3 else rng.randrange(1, n_max + 1)
        par = [-1] + [i - 1 if kind == 0 else (0 if kind == 1 else rng.randrange(0, i)) for i in range(1, n)]
        trees.append(par + [99] * (n_max - n))
        nodes.append(n)
    pos0 = [rng.randrange(0, 10 ** 6) for _ in trees]
    status = _status()
    out = st.rope_positions(_ints(pos0), parent=_ints(trees), n_nodes=_ints(nodes), dev_status=status)
    want = [[p + d for d in _depth(t, n)] + [-1] * (n_max - n) for p, t, n in zip(pos0, trees, nodes)]
    assert out.tolist() == want and int(status) == 0


def test_bad_trees_are_refused_alone():
    good = [-1, 0, 1, 1]
    trees = [good, [0, 0, 1, 1], [-1, 0, 2, 1], good, good, good]
    nodes, pos0 = [4, 4, 4, 0, 5, 4], [5, 5, 5, 5, 5, 2 ** 31 - 3]
    for b in range(1, 6):
        status = _status()
        pick = [0, b]
        out = st.rope_positions(_ints([pos0[i] for i in pick]), parent=_ints([trees[i] for i in pick]),
                                n_nodes=_ints([nodes[i] for i in pick]), dev_status=status)
        if b == 5:  # the deepest node sits at the largest position
            assert out.tolist()[1] == [2 ** 31 - 3, 2 ** 31 - 2, 2 ** 31 - 1, 2 ** 31 - 1] and int(status) == 0
        else:
            assert out.tolist() == [[5, 6, 7, 7], [-1] * 4] and int(status) == 4
    status = _status()
    out = st.rope_positions(_ints([2 ** 31 - 2]), parent=_ints([good]), n_nodes=_ints([4]), dev_status=status)
    assert out.tolist() == [[-1] * 4] and int(status) == 7


# ---- rotation ------------------------------------------------------------------------------------

def _rotated(x, positions, turns, layout, amplitude):
    """In 64 bits, and the magnitude of every pair."""
    rot = 2 * turns.numel()
    angle = (positions.long().reshape(-1, 1) * turns).double() * (2 * math.pi / 2.0 ** 64)  # wraps as the definition does
    c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    y = x.double().reshape(-1, *x.shape[-2:]).clone()
    i = torch.arange(rot // 2, device=x.device)
    lo, hi = (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)
    a, b = y[..., lo], y[..., hi]
    mag = torch.zeros_like(y)
    mag[..., lo] = mag[..., hi] = amplitude * torch.hypot(a, b)
    y[..., lo], y[..., hi] = amplitude * (a * c - b * s), amplitude * (a * s + b * c)
    return y.reshape(x.shape), mag.reshape(x.shape)


def _check(got, x, positions, turns, layout, amplitude=1.0):
    want, mag = _rotated(x, positions, turns, layout, amplitude)
    half = torch.finfo(x.dtype).eps / 2
    # an angle within pi 2^-32, cos and sin within 2^-23, the amplitude's product, two products and a sum, the last rounding
    bound = mag * (2.0 ** -30 + 6 * 2.0 ** -24) * 1.5 + half * want.abs() * (1 + half)
    bound = torch.where(mag > 0, bound, torch.zeros_like(bound) + (want != x.double()) * half * want.abs())
    assert ((got.double() - want).abs() <= bound).all(), ((got.double() - want).abs() - bound).max()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("n,hq,hk,d,rot", [(1, 32, 8, 128, 128), (1, 1, 1, 16, 16), (7, 3, 1, 48, 32), (300, 5, 5, 64, 48),
                                           (1001, 16, 2, 256, 240), (2100, 40, 8, 128, 64), (33, 64, 8, 64, 64)])
def test_rotation(dtype, layout, n, hq, hk, d, rot):
    gen = torch.Generator(device="cuda").manual_seed(n + d)
    q, k, _ = fused(gen, n, hq, hk, d, pad=1, dtype=dtype)
    pos = torch.randint(0, 2 ** 31 - 1, (n,), generator=gen, device="cuda", dtype=torch.int32)
    pos[0] = 2 ** 31 - 1
    turns = st.rope_table(rot, 10000.0).cuda()
    q_out, k_out = st.rope(q, k, pos, turns, layout=layout)
    assert q_out.is_contiguous() and k_out.is_contiguous()
    _check(q_out, q, pos, turns, layout)
    _check(k_out, k, pos, turns, layout)


def test_in_place_and_rows_without_a_position():
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = rows(gen, 50, 12, 64)
    q, k = x[:, :8], x[:, 8:10]
    before = x.clone()
    pos = torch.arange(50, device="cuda", dtype=torch.int32) - 10
    turns = st.rope_table(64, 500000.0).cuda()
    st.rope(q, k, pos, turns, q_out=q, k_out=k)
    assert torch.equal(x[:10], before[:10]) and torch.equal(x[:, 10:], before[:, 10:])
    _check(x[10:, :8], before[10:, :8], pos[10:], turns, "half")
    _check(x[10:, 8:10], before[10:, 8:10], pos[10:], turns, "half")


def test_amplitude_and_trees():
    gen = torch.Generator(device="cuda").manual_seed(4)
    q, k = rows(gen, 6 * 9, 4, 128, torch.float32), rows(gen, 6 * 9, 2, 128, torch.float32)
    q, k = q.view(6, 9, 4, 128), k.view(6, 9, 2, 128)
    pos = torch.randint(0, 100000, (6, 9), generator=gen, device="cuda", dtype=torch.int32)
    turns = st.rope_table(128, 10000.0, "ramp", 4.0, 4096, 1.0, 32.0).cuda()
    q_out, k_out = st.rope(q, k, pos, turns, amplitude=1.25)
    assert q_out.shape == q.shape and k_out.shape == k.shape
    _check(q_out, q, pos, turns, "half", 1.25)
    _check(k_out, k, pos, turns, "half", 1.25)


def test_relative_positions_at_far_places():
    """The product of a rotated query and key depends on their distance alone, wherever they are."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    q, k = rows(gen, 1, 1, 128, torch.float32), rows(gen, 1, 1, 128, torch.float32)
    turns = st.rope_table(128, 10000.0).cuda()

    def product(at, apart):
        a, _ = st.rope(q, k, _ints([at + apart]), turns)
        _, b = st.rope(q, k, _ints([at]), turns)
        return float((a.double() * b.double()).sum())

    size = float((q.double().norm() * k.double().norm()))
    for apart in (0, 1, 77, 5000):
        near = product(0, apart)
        for at in (10 ** 5, 10 ** 7, 2 ** 31 - 1 - apart):
            assert abs(product(at, apart) - near) <= size * 32 * 2.0 ** -24


def test_a_given_stream_and_a_captured_call():
    gen = torch.Generator(device="cuda").manual_seed(6)
    q, k = rows(gen, 40, 8, 128), rows(gen, 40, 2, 128)
    pos = torch.arange(40, device="cuda", dtype=torch.int32)
    turns = st.rope_table(128).cuda()
    want = st.rope(q, k, pos, turns)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = st.rope(q, k, pos, turns, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    q_out, k_out = torch.empty_like(q), torch.empty_like(k)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        st.rope(q, k, pos, turns, q_out=q_out, k_out=k_out)
    pos.add_(5)
    graph.replay()
    want = st.rope(q, k, pos, turns)
    assert torch.equal(q_out, want[0]) and torch.equal(k_out, want[1])
