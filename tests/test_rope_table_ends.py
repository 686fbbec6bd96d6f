"""Frequencies at the ends of their arguments, without a GPU."""

import math

import pytest

import tree_speculative_decoding_split_gb300 as st


@pytest.fixture(scope="module", autouse=True)
def built():
    st.build()


def _freq(turns):
    return [int(t) * 2.0 ** -64 * 2 * math.pi for t in turns]


def _near(g, w):
    return abs(g - w) <= 16 * 2.0 ** -52 * w + 2 * math.pi * 2.0 ** -64


@pytest.mark.parametrize("rot,base,length,low,high", [(128, 10000.0, 131072, 1.0, 32.0), (64, 10000.0, 1 << 20, 1.0, 4.0),
                                                     (128, 10000.0, 10 ** 9, 1.0, 32.0), (16, 100.0, 65536, 2.0, 500.0)])
def test_a_ramp_that_ends_behind_the_last_frequency(rot, base, length, low, high):
    """Where the lowest frequency still makes more than `low` turns over the trained length, the ramp goes on behind the last
    index: that frequency is weighted as its place on the ramp says, and kept where it makes more than `high`."""
    def index(r):
        return rot * math.log(length / (r * 2 * math.pi)) / (2 * math.log(base))

    hi, lo = max(math.floor(index(high)), 0), math.ceil(index(low))
    assert lo > rot // 2 - 1
    hi, lo = min(hi, rot - 1), min(lo, rot - 1)
    if lo == hi:
        lo += 0.001
    got = _freq(st.rope_table(rot, base, "ramp", 4.0, length, low, high))
    for i, g in enumerate(got):
        t, x = base ** (-2 * i / rot), min(max((i - hi) / (lo - hi), 0), 1)
        assert _near(g, t * (1 - x) + t / 4 * x)


@pytest.mark.parametrize("rot", [2 ** 32 + 64, 2 ** 33, -2 ** 32 + 64])
def test_sizes_past_32_bits_are_refused(rot):
    """(and not cut to their lower bits)"""
    with pytest.raises(st.SpecError) as e:
        st.rope_table(rot)
    assert e.value.code == 1


@pytest.mark.parametrize("length", [2 ** 64 + 8192, -2 ** 64 + 8192])
def test_lengths_past_64_bits(length):
    if length < 0:
        with pytest.raises(st.SpecError) as e:
            st.rope_table(64, scaling="bands", factor=8.0, original_len=length)
        assert e.value.code == 1
    else:  # (all frequencies turn often enough to be kept)
        got = st.rope_table(64, scaling="bands", factor=8.0, original_len=length)
        assert got.tolist() == st.rope_table(64).tolist()


@pytest.mark.parametrize("base,factor", [(1e300, 1e10), (10000.0, 1e308)])
def test_a_scaled_base_that_is_not_finite_is_refused(base, factor):
    with pytest.raises(st.SpecError) as e:
        st.rope_table(64, base, "base", factor)
    assert e.value.code == 1
