"""Pins of the 8-bit cache's oracle: the number format against torch's own float8 type and hand values,
the scale rule, appending across block borders, and the block stack against a hand example."""

import numpy as np
import torch

import oracle


def test_decode_and_encode_against_torch():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(oracle.E4M3, want, equal_nan=True)
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.standard_normal(20000) * 2.0 ** rng.integers(-12, 9, 20000), (want[:126] + want[1:127]) / 2])
    x = x[np.abs(x) <= 448].astype(np.float32)
    got = oracle.e4m3_encode(x)
    ref = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(oracle.E4M3[got], oracle.E4M3[ref])


def test_saturation_and_nan():
    got = oracle.E4M3[oracle.e4m3_encode([1e9, -np.inf, 449.0, np.nan, 2.0 ** -10, 2.0 ** -11, 3 * 2.0 ** -10])]
    assert np.array_equal(got, [448, -448, 448, np.nan, 0, 0, 2.0 ** -8], equal_nan=True)  # ties to even


def test_scale_rule():
    assert oracle.block_scale([448.0]) == 1 and oracle.block_scale([448.5]) == 2
    assert oracle.block_scale([1.75]) == 2.0 ** -8 and oracle.block_scale([1.0, np.inf, np.nan]) == 2.0 ** -8
    assert oracle.block_scale([0.0]) == 2.0 ** -64 and oracle.block_scale([3e38]) == 2.0 ** 120
    for top in np.abs(np.random.default_rng(1).standard_normal(200)) * 100:
        s = oracle.block_scale([top])
        assert top <= 448 * s and top > 448 * s / 2 and np.log2(s) % 1 == 0


def test_append_across_a_border():
    cache, scale = np.zeros((3, 1, 2, 1), np.uint8), np.ones((3, 1))
    rows = np.array([1.0, 2.0, 1000.0]).reshape(3, 1, 1)
    oracle.append_rows(rows[:1], cache, scale, 0, [2, 0], 2)
    assert scale[2, 0] == 2.0 ** -8
    oracle.append_rows(rows[1:], cache, scale, 1, [2, 0], 2)
    assert scale[2, 0] == 2.0 ** -7 and scale[0, 0] == 4  # 2 needs a larger scale; 1000 <= 448 * 4
    assert oracle.gather_kv8(cache, scale, [2, 0], 2, 3)[0, :, 0].tolist() == [1, 2, 1024]


def test_reserve_hand_example():
    table, free = [[5], [7, 8, 9]], [1, 2, 3]
    slots = oracle.reserve([3, 4], [6, 0], table, free, 4)  # wants 3 and 1 blocks
    # 8 and 9 are given back (8 on top), then request 0 takes two from the top
    assert table == [[5, 8, 9], [7]] and free == [1, 2, 3]
    assert slots[0] == [5 * 4 + 3, 32, 33, 34, 35, 36] and slots[1] == []
    table, free = [[], [0], []], [4]
    slots = oracle.reserve([0, 1, 0], [5, 1, 0], table, free, 4)
    assert slots[0] is None and table == [[], [0], []] and slots[1] == [1] and slots[2] == []


def test_growth_then_shrinking_restores_the_stack():
    rng = np.random.default_rng(2)
    order = rng.permutation(40).tolist()
    table, free = [order[:3], order[3:4], []], order[4:]
    before = ([list(t) for t in table], list(free))
    oracle.reserve([40, 10, 0], [33, 70, 100], table, free, 16)
    oracle.reserve([40, 10, 0], [0, 0, 0], table, free, 16)
    assert (table, free) == before
