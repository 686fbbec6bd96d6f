"""Positions of rows of no request: refusals of the field that asks for them, without a GPU."""

import ctypes

import pytest

import tree_speculative_decoding_split_gb300 as st

FAKE = ctypes.c_void_p(1 << 20)


@pytest.fixture(scope="module")
def L():
    st.build()
    return st.lib()


@pytest.mark.parametrize("kw", [dict(fill=2), dict(fill=-1), dict(reserved0=1),
                                dict(fill=1, row_start=None, parent=FAKE, n_nodes=FAKE, n_rows=0, n_max=9)])
def test_refused_fills(L, kw):
    a = dict(batch=2, n_max=0, n_rows=10, pos0=FAKE, row_start=FAKE, positions=FAKE)
    a.update(kw)
    assert L.spec_rope_positions(ctypes.byref(st.RopePositionsArgs(**a)), None, None) == 1
