"""The prompt calls' host side, without a GPU: frequencies, struct layouts, refusals before any launch."""

import ctypes
import math
import os
import subprocess
import tempfile

import pytest
import torch

import tree_speculative_decoding_split_gb300 as st

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = ctypes.c_void_p(1 << 20)


@pytest.fixture(scope="module")
def L():
    st.build()
    return st.lib()


def _freq(turns):
    return [int(t) * 2.0 ** -64 * 2 * math.pi for t in turns]


def _theta(rot, base):
    return [base ** (-2 * i / rot) for i in range(rot // 2)]


def _near(got, want):
    # the frequencies in 64 bits: pow and a few products, and 2^-64 of a turn cut off
    return all(abs(g - w) <= 16 * 2.0 ** -52 * w + 2 * math.pi * 2.0 ** -64 for g, w in zip(got, want))


@pytest.mark.parametrize("rot", [2, 16, 64, 128, 256])
@pytest.mark.parametrize("base", [2.0, 10000.0, 500000.0])
def test_plain_linear_and_base_frequencies(L, rot, base):
    theta = _theta(rot, base)
    turns = st.rope_table(rot, base)
    assert turns.dtype == torch.int64 and turns.shape == (rot // 2,) and not turns.is_cuda
    assert _near(_freq(turns), theta)
    assert _near(_freq(st.rope_table(rot, base, "linear", 8.0)), [t / 8 for t in theta])
    if rot > 2:
        assert _near(_freq(st.rope_table(rot, base, "base", 4.0)), _theta(rot, base * 4.0 ** (rot / (rot - 2))))


def test_frequency_bands(L):
    theta = _theta(128, 500000.0)
    got = _freq(st.rope_table(128, 500000.0, "bands", 8.0, 8192, 1.0, 4.0))
    kinds = set()
    for t, g in zip(theta, got):
        r = 8192 * t / (2 * math.pi)
        if r >= 4:
            want, kind = t, "kept"
        elif r <= 1:
            want, kind = t / 8, "scaled"
        else:
            x = (r - 1) / 3
            want, kind = (1 - x) * t / 8 + x * t, "between"
        kinds.add(kind)
        assert _near([g], [want])
    assert kinds == {"kept", "scaled", "between"}


@pytest.mark.parametrize("rot,base,length,low,high", [(128, 10000.0, 4096, 1.0, 32.0), (64, 500000.0, 8192, 2.0, 3.0),
                                                     (16, 10000.0, 100, 1.0, 32.0), (64, 10000.0, 4096, 1.0, 1.001)])
def test_frequency_ramp(L, rot, base, length, low, high):
    theta = _theta(rot, base)
    got = _freq(st.rope_table(rot, base, "ramp", 4.0, length, low, high))

    def index(r):
        return rot * math.log(length / (r * 2 * math.pi)) / (2 * math.log(base))

    top = rot // 2 - 1
    hi = min(max(math.floor(index(high)), 0), top)
    lo = max(min(max(math.ceil(index(low)), 0), top), hi + 0.001)
    for i, (t, g) in enumerate(zip(theta, got)):
        x = min(max((i - hi) / (lo - hi), 0), 1)
        assert _near([g], [t * (1 - x) + t / 4 * x])


@pytest.mark.parametrize("kwargs,code", [
    (dict(rot_dim=0), 1), (dict(rot_dim=3), 1), (dict(rot_dim=64, base=1.0), 1), (dict(rot_dim=64, base=math.nan), 1),
    (dict(rot_dim=64, scaling="linear", factor=0.0), 1), (dict(rot_dim=64, scaling="linear", factor=math.inf), 1),
    (dict(rot_dim=64, scaling="bands", factor=8.0, original_len=0), 1),
    (dict(rot_dim=64, scaling="bands", factor=8.0, original_len=8192, low=4.0, high=4.0), 1),
    (dict(rot_dim=64, scaling="ramp", factor=8.0, original_len=8192, low=0.0, high=4.0), 1),
    (dict(rot_dim=2, scaling="base", factor=2.0), 1), (dict(rot_dim=64, scaling="linear", factor=0.1), 2)])
def test_refused_frequencies(L, kwargs, code):
    with pytest.raises(st.SpecError) as e:
        st.rope_table(**kwargs)
    assert e.value.code == code


def test_a_refused_table_writes_nothing(L):
    turns = (ctypes.c_int64 * 32)(*([7] * 32))
    assert L.spec_rope_table(64, 10000.0, 1, 0.1, 0, 0.0, 0.0, turns) == 2 and list(turns) == [7] * 32
    assert L.spec_rope_table(64, 10000.0, 9, 1.0, 0, 0.0, 0.0, turns) == 2
    assert L.spec_rope_table(64, 10000.0, 0, 1.0, 0, 0.0, 0.0, None) == 1


def test_struct_layouts_match_the_header():
    structs = {"spec_rope_positions_args": st.RopePositionsArgs, "spec_rope_args": st.RopeArgs,
               "spec_prompt_attn_args": st.PromptAttnArgs, "spec_key_weights_args": st.KeyWeightsArgs,
               "spec_kv_keep_args": st.KvKeepArgs}
    lines = []
    for name, cls in structs.items():
        lines.append(f'printf("{name} size %zu\\n", sizeof({name}));')
        lines += [f'printf("{name} {f[0]} %zu\\n", offsetof({name}, {f[0]}));' for f in cls._fields_]
    src = "#include <stddef.h>\n#include <stdio.h>\n#include \"spectree.h\"\nint main(void) {" + "\n".join(lines) + "return 0;}"
    with tempfile.TemporaryDirectory() as td:
        c, exe = os.path.join(td, "l.c"), os.path.join(td, "l")
        open(c, "w").write(src)
        subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), c, "-o", exe], check=True)
        out = subprocess.run([exe], capture_output=True, text=True, check=True).stdout
    for line in out.splitlines():
        name, field, at = line.split()
        cls = structs[name]
        assert (ctypes.sizeof(cls) if field == "size" else getattr(cls, field).offset) == int(at), line


def _positions(**kw):
    a = dict(batch=2, n_max=0, n_rows=10, pos0=FAKE, row_start=FAKE, positions=FAKE)
    a.update(kw)
    return st.RopePositionsArgs(**a)


def _rope(**kw):
    a = dict(dtype=1, layout=0, num_q_heads=8, num_k_heads=2, head_dim=64, rot_dim=64, n_rows=10, q_stride=512, k_stride=128,
             q_out_stride=512, k_out_stride=128, amplitude=1.0, q=FAKE, k=FAKE, positions=FAKE, turns=FAKE,
             q_out=ctypes.c_void_p(1 << 21), k_out=ctypes.c_void_p(1 << 21))
    a.update(kw)
    return st.RopeArgs(**a)


def _attn(**kw):
    a = dict(dtype=1, batch=2, num_q_heads=8, num_kv_heads=2, head_dim=64, n_rows=10, q_stride=512, k_stride=128, v_stride=128,
             q=FAKE, k=FAKE, v=FAKE, row_start=FAKE, out=FAKE)
    a.update(kw)
    return st.PromptAttnArgs(**a)


def _weights(**kw):
    a = dict(dtype=1, batch=2, num_q_heads=8, num_kv_heads=2, head_dim=64, window=4, n_rows=10, q_stride=512, k_stride=128,
             q=FAKE, k=FAKE, lse=FAKE, row_start=FAKE, weight=FAKE)
    a.update(kw)
    return st.KeyWeightsArgs(**a)


def _keep(**kw):
    a = dict(dtype=1, batch=2, num_kv_heads=2, head_dim=64, budget=5, first=1, last=2, n_rows=10, rows_out=10, k_stride=128,
             v_stride=128, k=FAKE, v=FAKE, weight=FAKE, row_start=FAKE, k_out=FAKE, v_out=FAKE, index=FAKE, keep_start=FAKE,
             n_keep=FAKE)
    a.update(kw)
    return st.KvKeepArgs(**a)


ODD = ctypes.c_void_p((1 << 20) + 8)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), 1), (dict(pos0=None), 1), (dict(row_start=None), 1), (dict(parent=FAKE), 1), (dict(n_nodes=FAKE), 1),
    (dict(n_rows=-1), 1), (dict(positions=None), 1), (dict(n_max=3), 1), (dict(n_rows=1 << 31), 2), (dict(batch=8193), 2),
    (dict(row_start=None, parent=FAKE, n_nodes=FAKE, n_rows=0, n_max=256), 2),
    (dict(row_start=None, parent=FAKE, n_nodes=FAKE, n_rows=0, n_max=0), 1),
    (dict(row_start=None, parent=FAKE, n_nodes=FAKE, n_rows=5, n_max=9), 1), (dict(row_start=None, parent=FAKE, n_rows=0, n_max=9), 1)])
def test_refused_positions(L, kw, code):
    assert L.spec_rope_positions(ctypes.byref(_positions(**kw)), None, None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), 2), (dict(layout=2), 2), (dict(head_dim=72, rot_dim=64), 2), (dict(head_dim=272), 2), (dict(rot_dim=8), 2),
    (dict(rot_dim=80), 2), (dict(num_q_heads=0), 1), (dict(num_k_heads=0), 1), (dict(n_rows=-1), 1), (dict(n_rows=1 << 31), 2),
    (dict(q_stride=511), 1), (dict(q_stride=516), 1), (dict(k_out_stride=64), 1), (dict(amplitude=math.nan), 1),
    (dict(amplitude=math.inf), 1), (dict(reserved0=1), 1), (dict(q=None), 1), (dict(turns=None), 1), (dict(positions=None), 1),
    (dict(q=ODD), 1), (dict(k_out=ODD), 1), (dict(q_out=FAKE, q_out_stride=520), 1), (dict(num_q_heads=65535, q_stride=1 << 30), 2)])
def test_refused_rotations(L, kw, code):
    assert L.spec_rope(ctypes.byref(_rope(**kw)), None) == code


SHARED = [(dict(dtype=0), 2), (dict(head_dim=96), 2), (dict(batch=0), 1), (dict(batch=8193), 2), (dict(num_q_heads=9), 1),
          (dict(num_kv_heads=0), 1), (dict(num_q_heads=258, q_stride=258 * 64), 2), (dict(n_rows=-1), 1),
          (dict(n_rows=(1 << 31) - 256), 2), (dict(q_stride=508), 1), (dict(q_stride=448), 1), (dict(k_stride=1 << 38), 1),
          (dict(scale=math.nan), 1), (dict(q=None), 1), (dict(k=ODD), 1), (dict(row_start=None), 1)]


@pytest.mark.parametrize("kw,code", SHARED + [(dict(v=None), 1), (dict(out=ODD), 1), (dict(v_stride=64), 1)])
def test_refused_prompt_attention(L, kw, code):
    a = ctypes.byref(_attn(**kw))
    assert L.spec_prompt_attention_workspace(a) == 0
    assert L.spec_prompt_attention(a, FAKE, 1 << 30, None, None) == code


@pytest.mark.parametrize("kw,code", SHARED + [(dict(window=0), 1), (dict(lse=None), 1), (dict(weight=None), 1), (dict(reserved0=2), 1)])
def test_refused_key_weights(L, kw, code):
    a = ctypes.byref(_weights(**kw))
    assert L.spec_prompt_key_weights_workspace(a) == 0
    assert L.spec_prompt_key_weights(a, FAKE, 1 << 30, None, None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=3), 2), (dict(head_dim=32), 2), (dict(batch=0), 1), (dict(batch=8193), 2), (dict(num_kv_heads=0), 1),
    (dict(budget=0), 1), (dict(first=-1), 1), (dict(last=-1), 1), (dict(first=3, last=3), 1), (dict(n_rows=-1), 1),
    (dict(rows_out=-1), 1), (dict(n_rows=1 << 31), 2), (dict(n_rows=(1 << 31) - 16384), 2), (dict(rows_out=1 << 31), 2), (dict(k_stride=120), 1), (dict(v_stride=132), 1),
    (dict(k=None), 1), (dict(v=ODD), 1), (dict(weight=None), 1), (dict(row_start=None), 1), (dict(index=None), 1),
    (dict(keep_start=None), 1), (dict(n_keep=None), 1), (dict(reserved0=1), 1),
    (dict(batch=8192, num_kv_heads=1 << 15, k_stride=1 << 21, v_stride=1 << 21), 2)])
def test_refused_kv_keep(L, kw, code):
    a = ctypes.byref(_keep(**kw))
    assert L.spec_kv_keep_workspace(a) == 0
    assert L.spec_kv_keep(a, FAKE, 1 << 30, None, None) == code


def test_workspaces(L):
    for name, args in (("spec_prompt_attention", _attn()), ("spec_prompt_key_weights", _weights()), ("spec_kv_keep", _keep())):
        a = ctypes.byref(args)
        call, need = getattr(L, name), getattr(L, name + "_workspace")(a)
        assert need > 0
        assert call(a, None, need, None, None) == 1
        assert call(a, ODD, need, None, None) == 1
        assert call(a, FAKE, need - 1, None, None) == 3
        assert call(None, FAKE, need, None, None) == 1


def test_tensors_on_the_host_are_refused():
    q, k = torch.zeros((4, 8, 64), dtype=torch.bfloat16), torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    ints = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        st.rope_positions(ints, row_start=torch.zeros(4, dtype=torch.int32), n_rows=4)
    with pytest.raises(ValueError):
        st.rope(q, k, ints, torch.zeros(32, dtype=torch.int64))
    with pytest.raises(ValueError):
        st.prompt_attention(q, k, k, ints)
    with pytest.raises(ValueError):
        st.prompt_key_weights(q, k, torch.zeros((4, 8)), ints, 4)
    with pytest.raises(ValueError):
        st.kv_keep(k, k, torch.zeros((2, 4)), ints, 4)
