"""Host side of the 8-bit paged cache's calls, without a GPU: struct layouts against the header, and
arguments that are refused before anything is launched."""

import ctypes
import os
import subprocess

import pytest

import tree_speculative_decoding_split_gb300 as st

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 20  # a 16-byte aligned address that nothing reads: every call here is refused


@pytest.fixture(scope="module")
def L():
    st.build()
    return st.lib()


def test_struct_layouts_match_the_header(tmp_path):
    structs = (("spec_kv_reserve_args", st.KvReserveArgs), ("spec_kv8_append_args", st.Kv8AppendArgs),
               ("spec_attn_kv8_args", st.AttnKv8Args))
    lines = ["#include <stddef.h>", "#include <stdio.h>", '#include "spectree.h"', "int main(void) {"]
    for name, cls in structs:
        lines.append(f'printf("{name} %zu\\n", sizeof({name}));')
        lines += [f'printf("{name}.{f} %zu\\n", offsetof({name}, {f}));' for f, _ in cls._fields_]
    (tmp_path / "l.c").write_text("\n".join(lines + ["return 0; }"]))
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(tmp_path / "l.c"), "-o",
                    str(tmp_path / "l")], check=True)
    got = dict(line.split() for line in subprocess.run([str(tmp_path / "l")], capture_output=True, text=True,
                                                       check=True).stdout.splitlines())
    for name, cls in structs:
        assert int(got[name]) == ctypes.sizeof(cls)
        for f, _ in cls._fields_:
            assert int(got[f"{name}.{f}"]) == getattr(cls, f).offset, (name, f)


def _reserve(**kw):
    a = dict(batch=2, block_size=16, max_blocks=8, num_blocks=32, slot_cap=64, seq_len=P, n_new=P, block_table=P,
             n_blocks=P, free_list=P, free_count=P, slot_map=P, row_start=P)
    a.update(kw)
    return st.KvReserveArgs(**a)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), 1), (dict(slot_cap=-1), 1), (dict(block_size=24), 2), (dict(max_blocks=0), 1),
    (dict(num_blocks=0), 1), (dict(batch=8193), 2), (dict(slot_cap=1 << 31), 2), (dict(seq_len=None), 1),
    (dict(n_new=None), 1), (dict(block_table=None), 1), (dict(n_blocks=None), 1), (dict(free_list=None), 1),
    (dict(free_count=None), 1), (dict(row_start=None), 1), (dict(slot_map=P + 8), 1),
    (dict(batch=8192, max_blocks=1 << 18), 2)])
def test_reserve_refusals(L, kw, code):
    assert L.spec_kv_reserve(ctypes.byref(_reserve(**kw)), None, None) == code


def _append(**kw):
    a = dict(dtype=1, batch=2, num_kv_heads=2, head_dim=128, block_size=16, max_blocks=8, num_blocks=32, n_max=0,
             path_cap=0, reserved0=0, n_rows=40, k_new=P, v_new=P, row_start=P, path=None, accept_len=None, seq_len=P,
             block_table=P, k_cache=P, v_cache=P, k_scale=P, v_scale=P, new_len=2 * P)
    a.update(kw)
    return st.Kv8AppendArgs(**a)


_PATH = dict(path=P, accept_len=P, row_start=None, n_rows=0, n_max=63, path_cap=6)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), 2), (dict(batch=0), 1), (dict(num_kv_heads=0), 1), (dict(head_dim=96), 2), (dict(block_size=8), 2),
    (dict(max_blocks=0), 1), (dict(num_blocks=1 << 30), 2), (dict(reserved0=1), 1), (dict(n_rows=-1), 1),
    (dict(n_rows=1 << 31), 2), (dict(k_new=None), 1), (dict(v_new=P + 4), 1), (dict(row_start=None), 1),
    (dict(accept_len=P), 1), (dict(n_max=3), 1), (dict(path_cap=3), 1), (dict(seq_len=None), 1), (dict(new_len=P), 1),
    (dict(block_table=None), 1), (dict(k_cache=P + 1), 1), (dict(v_cache=None), 1), (dict(k_scale=None), 1),
    (dict(v_scale=None), 1), (dict(_PATH, accept_len=None), 1), (dict(_PATH, row_start=P), 1), (dict(_PATH, n_rows=3), 1),
    (dict(_PATH, n_max=0), 1), (dict(_PATH, n_max=256), 2), (dict(_PATH, path_cap=0), 1),
    (dict(n_rows=(1 << 31) - 1, batch=(1 << 31) - 1), 2)])
def test_append_refusals(L, kw, code):
    assert L.spec_kv8_append(ctypes.byref(_append(**kw)), None, None) == code


def _attn(**kw):
    a = dict(dtype=1, batch=2, n_max=5, num_q_heads=8, num_kv_heads=2, head_dim=128, block_size=16, max_blocks=64,
             num_blocks=256, scale=0.0, q=P, k_tree=P, v_tree=P, k_cache=P, v_cache=P, k_scale=P, v_scale=P,
             prefix_len=P, n_nodes=P, parent=P, block_table=P, out=P, lse=P)
    a.update(kw)
    return st.AttnKv8Args(**a)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=0), 2), (dict(batch=0), 1), (dict(n_max=0), 1), (dict(n_max=256), 2), (dict(num_q_heads=7), 1),
    (dict(head_dim=256), 2), (dict(block_size=48), 2), (dict(max_blocks=0), 1), (dict(num_blocks=0), 1),
    (dict(max_blocks=1 << 27), 2), (dict(batch=40000), 2), (dict(num_q_heads=514), 2), (dict(q=None), 1), (dict(k_tree=P + 2), 1),
    (dict(v_tree=None), 1), (dict(k_cache=None), 1), (dict(v_cache=P + 8), 1), (dict(k_scale=None), 1),
    (dict(v_scale=None), 1), (dict(prefix_len=None), 1), (dict(n_nodes=None), 1), (dict(parent=None), 1),
    (dict(block_table=None), 1), (dict(out=P + 8), 1)])
def test_attention_refusals(L, kw, code):
    a = _attn(**kw)
    assert L.spec_tree_attention_kv8_workspace(ctypes.byref(a)) == 0
    assert L.spec_tree_attention_kv8(ctypes.byref(a), P, 1 << 40, None, None) == code


def test_attention_workspace_refusals(L):
    a = _attn()
    need = L.spec_tree_attention_kv8_workspace(ctypes.byref(a))
    assert need > 0
    assert L.spec_tree_attention_kv8(ctypes.byref(a), None, need, None, None) == 1
    assert L.spec_tree_attention_kv8(ctypes.byref(a), P + 8, need, None, None) == 1
    assert L.spec_tree_attention_kv8(ctypes.byref(a), P, need - 1, None, None) == 3


def test_null_structs(L):
    assert L.spec_kv_reserve(None, None, None) == 1
    assert L.spec_kv8_append(None, None, None) == 1
    assert L.spec_tree_attention_kv8(None, None, 0, None, None) == 1
    assert L.spec_tree_attention_kv8_workspace(None) == 0


def test_binding_refuses_host_tensors():
    import torch
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        st.kv_reserve(i, i, torch.zeros((2, 4), dtype=torch.int32), i, i, i[:1], 16)
    x = torch.zeros((2, 1, 2, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        st.tree_attention_kv8(x, x, x, x, x, x, x, i, i, i, i)
    with pytest.raises(ValueError):
        st.kv8_append(x, x, x, x, x, x, i, i)
