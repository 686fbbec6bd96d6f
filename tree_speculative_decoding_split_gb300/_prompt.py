"""Binding of the calls that take prompts to the cache: argument structs, checks and launches.

    rope_table(...)          frequencies for rope, with the scalings of long contexts (host)
    rope_positions(...)      positions of packed prompt rows or tree nodes
    rope(...)                rotary positions of q and k
    prompt_attention(...)    causal attention over packed prompts
    prompt_key_weights(...)  attention weight of every key from each prompt's last rows
    kv_keep(...)             the rows that a budget leaves, packed for kv8_append

As for the 8-bit cache's calls, the plain call is marshalled natively (``csrc/marshal.cpp``); any other, and
every refused one, goes through the functions here.
"""

import ctypes

from . import (_answer, _check, _dtype_code, _fast, _launch, _native, _need, _status_ptr, _torch, _vp, _workspace, lib)

ROPE_KINDS = {"none": 0, "linear": 1, "base": 2, "bands": 3, "ramp": 4}
ROPE_LAYOUTS = {"half": 0, "interleaved": 1}

_i32, _i64, _f32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_float


class RopePositionsArgs(ctypes.Structure):
    _fields_ = [("batch", _i32), ("n_max", _i32), ("n_rows", _i64), ("pos0", _vp), ("row_start", _vp), ("parent", _vp),
                ("n_nodes", _vp), ("positions", _vp), ("fill", _i32), ("reserved0", _i32)]


class RopeArgs(ctypes.Structure):
    _fields_ = [("dtype", _i32), ("layout", _i32), ("num_q_heads", _i32), ("num_k_heads", _i32), ("head_dim", _i32),
                ("rot_dim", _i32), ("n_rows", _i64), ("q_stride", _i64), ("k_stride", _i64), ("q_out_stride", _i64),
                ("k_out_stride", _i64), ("amplitude", _f32), ("reserved0", _i32), ("q", _vp), ("k", _vp), ("positions", _vp),
                ("turns", _vp), ("q_out", _vp), ("k_out", _vp)]


class PromptAttnArgs(ctypes.Structure):
    _fields_ = [("dtype", _i32), ("batch", _i32), ("num_q_heads", _i32), ("num_kv_heads", _i32), ("head_dim", _i32),
                ("scale", _f32), ("n_rows", _i64), ("q_stride", _i64), ("k_stride", _i64), ("v_stride", _i64), ("q", _vp),
                ("k", _vp), ("v", _vp), ("row_start", _vp), ("out", _vp), ("lse", _vp)]


class KeyWeightsArgs(ctypes.Structure):
    _fields_ = [("dtype", _i32), ("batch", _i32), ("num_q_heads", _i32), ("num_kv_heads", _i32), ("head_dim", _i32),
                ("scale", _f32), ("window", _i32), ("reserved0", _i32), ("n_rows", _i64), ("q_stride", _i64), ("k_stride", _i64),
                ("q", _vp), ("k", _vp), ("lse", _vp), ("row_start", _vp), ("weight", _vp)]


class KvKeepArgs(ctypes.Structure):
    _fields_ = [("dtype", _i32), ("batch", _i32), ("num_kv_heads", _i32), ("head_dim", _i32), ("budget", _i32), ("first", _i32),
                ("last", _i32), ("reserved0", _i32), ("n_rows", _i64), ("rows_out", _i64), ("k_stride", _i64),
                ("v_stride", _i64), ("k", _vp), ("v", _vp), ("weight", _vp), ("row_start", _vp), ("k_out", _vp), ("v_out", _vp),
                ("index", _vp), ("keep_start", _vp), ("n_keep", _vp)]


def declare(L):
    """Argument and result types of these calls (called once by the package's ``lib``)."""
    L.spec_rope_table.argtypes = [_i32, ctypes.c_double, _i32, ctypes.c_double, _i64, ctypes.c_double, ctypes.c_double,
                                  ctypes.POINTER(_i64)]
    L.spec_rope_table.restype = _i32
    L.spec_rope_positions.argtypes = [ctypes.POINTER(RopePositionsArgs), _vp, _vp]
    L.spec_rope_positions.restype = _i32
    L.spec_rope.argtypes = [ctypes.POINTER(RopeArgs), _vp]
    L.spec_rope.restype = _i32
    for name, args in (("spec_prompt_attention", PromptAttnArgs), ("spec_prompt_key_weights", KeyWeightsArgs),
                       ("spec_kv_keep", KvKeepArgs)):
        size, call = getattr(L, name + "_workspace"), getattr(L, name)
        size.argtypes = [ctypes.POINTER(args)]
        size.restype = ctypes.c_size_t
        call.argtypes = [ctypes.POINTER(args), _vp, ctypes.c_size_t, _vp, _vp]
        call.restype = _i32


def _rows(t, name, dtype, dev):
    """(address, rows, heads, head_dim, elements between rows) of rows of heads [...][H][d], possibly a view of wider
    rows: the heads of a row lie together, the rows at one distance."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must live on a CUDA device")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() < 3:
        raise ValueError(f"{name} must be rows of heads [...][H][d]")
    shape, strides = t.shape, t.stride()
    H, d = shape[-2:]
    if (d > 1 and strides[-1] != 1) or (H > 1 and strides[-2] != d):
        raise ValueError(f"the heads of a row of {name} must lie together")
    rows, step = 1, None
    for n, s in zip(reversed(shape[:-2]), reversed(strides[:-2])):
        if n > 1:
            if step is None:
                step = s
            elif s != step * rows:
                raise ValueError(f"the rows of {name} must lie at one distance")
        rows *= n
    return t.data_ptr(), rows, H, d, H * d if step is None else step


def _clip(x, bits=32):
    """x for a field of 32 (64) bits: what lies outside is as good as its nearer end (and would be cut to its lower bits)."""
    return max(-2 ** (bits - 1), min(int(x), 2 ** (bits - 1) - 1))


def _on(dev, fn, *args):
    """fn(*args) with dev current (sizes go by the current device)."""
    torch = _torch()
    with torch.cuda.device(dev):
        return fn(*args)


def rope_table(rot_dim, base=10000.0, scaling="none", factor=1.0, original_len=0, low=1.0, high=4.0):
    """Rotary frequencies as 2^-64 turns per position (see spec_rope_table): an int64 CPU tensor [rot_dim / 2].
    ``scaling``: "none", "linear", "base", "bands" or "ramp"."""
    torch = _torch()
    rot = _clip(rot_dim)  # (odd where it was past 32 bits: refused, with nothing to hold)
    turns = torch.empty(1 if rot % 2 else max(rot // 2, 1), dtype=torch.int64)
    code = lib().spec_rope_table(rot, float(base), ROPE_KINDS[scaling], float(factor), _clip(original_len, 64), float(low),
                                 float(high), ctypes.cast(turns.data_ptr(), ctypes.POINTER(_i64)))
    _check(code, "spec_rope_table")
    return turns


def rope_positions_args(pos0, row_start=None, n_rows=None, parent=None, n_nodes=None, positions=None):
    """Build the C argument struct for rope_positions (tensors are validated here); returns (args, positions)."""
    torch = _torch()
    i32 = torch.int32
    _need(pos0, "pos0", i32)
    dev, B = pos0.device, pos0.numel()
    ix = dev.index
    if (row_start is None) == (parent is None):
        raise ValueError("positions are those of packed rows (row_start) or of trees (parent)")
    if parent is not None:
        if n_rows is not None or n_nodes is None:
            raise ValueError("parent [B][N] goes with n_nodes [B] and no n_rows")
        source = (None, _fast(parent, "parent", i32, dev, ix), _fast(n_nodes, "n_nodes", i32, dev, ix))
        if parent.dim() != 2 or parent.shape[0] != B or n_nodes.numel() != B:
            raise ValueError("parent must be [B][N], n_nodes and pos0 [B]")
        shape, N, rows = tuple(parent.shape), parent.shape[1], 0
    else:
        if n_nodes is not None or (n_rows is None and positions is None):
            raise ValueError("row_start [B + 1] goes with n_rows or positions, and no n_nodes")
        source = (_fast(row_start, "row_start", i32, dev, ix), None, None)
        if row_start.numel() != B + 1:
            raise ValueError("row_start must be [B + 1], pos0 [B]")
        rows = positions.numel() if n_rows is None else int(n_rows)
        shape, N = (rows,), 0
    fill = int(positions is None and parent is None)
    if positions is None:
        positions = torch.empty(shape, dtype=i32, device=dev)
    elif tuple(positions.shape) != shape:
        raise ValueError("positions must be [n_rows], or [B][N] for trees")
    a = RopePositionsArgs(B, N, rows, pos0.data_ptr(), *source, _fast(positions, "positions", i32, dev, ix), fill, 0)
    return a, positions


def rope_positions(pos0, row_start=None, n_rows=None, parent=None, n_nodes=None, positions=None, dev_status=None,
                   stream=None):
    """Positions of packed prompt rows (``row_start`` [B + 1], ``n_rows``) or of tree nodes (``parent`` [B][N],
    ``n_nodes``), int32 (see spec_rope_positions).  Rows of no request, all of them where row_start is refused, have
    position -1; in ``positions`` of the caller's own they keep what it holds."""
    if stream is None:
        r = _native().positions(pos0, row_start, n_rows, parent, n_nodes, positions, dev_status)
        if r is not None:
            return _answer(r, "spec_rope_positions")
    a, positions = rope_positions_args(pos0, row_start, n_rows, parent, n_nodes, positions)
    _launch(lib().spec_rope_positions, "spec_rope_positions", pos0.device, stream, (positions,), ctypes.byref(a),
            _status_ptr(dev_status, pos0.device))
    return positions


def rope_args(q, k, positions, turns, layout="half", amplitude=1.0, q_out=None, k_out=None):
    """Build the C argument struct for rope (tensors are validated here); returns (args, q_out, k_out)."""
    torch = _torch()
    if not isinstance(q, torch.Tensor):
        raise TypeError("q must be a torch.Tensor")
    dev, dtype = q.device, q.dtype
    ix = dev.index
    code = _dtype_code(q)
    q_ptr, rows, Hq, d, q_step = _rows(q, "q", dtype, dev)
    k_ptr, k_rows, Hk, k_d, k_step = _rows(k, "k", dtype, dev)
    pos = _fast(positions, "positions", torch.int32, dev, ix)
    freq = _fast(turns, "turns", torch.int64, dev, ix)
    if k_rows != rows or k_d != d or positions.numel() != rows:
        raise ValueError("q and k must be [...][H][d] with a position for each row")
    if q_out is None:
        q_out = torch.empty(q.shape, dtype=dtype, device=dev)
    if k_out is None:
        k_out = torch.empty(k.shape, dtype=dtype, device=dev)
    if q_out.shape != q.shape or k_out.shape != k.shape:
        raise ValueError("q_out and k_out must have the shapes of q and k")
    qo_ptr, _, _, _, qo_step = _rows(q_out, "q_out", dtype, dev)
    ko_ptr, _, _, _, ko_step = _rows(k_out, "k_out", dtype, dev)
    a = RopeArgs(code, ROPE_LAYOUTS[layout], Hq, Hk, d, 2 * turns.numel(), rows, q_step, k_step, qo_step, ko_step,
                 float(amplitude), 0, q_ptr, k_ptr, pos, freq, qo_ptr, ko_ptr)
    return a, q_out, k_out


def rope(q, k, positions, turns, layout="half", amplitude=1.0, q_out=None, k_out=None, stream=None):
    """Rotary positions of q [...][Hq][d] and k [...][Hkv][d] by one position per row and the frequencies ``turns``
    (int64 [rot_dim / 2], see rope_table and spec_rope).  Rows with a negative position are not written.  ``q_out=q,
    k_out=k`` works in place.  Returns (q_out, k_out)."""
    if stream is None:
        r = _native().rope(q, k, positions, turns, ROPE_LAYOUTS[layout], amplitude, q_out, k_out)
        if r is not None:
            return _answer(r, "spec_rope")
    a, q_out, k_out = rope_args(q, k, positions, turns, layout, amplitude, q_out, k_out)
    _launch(lib().spec_rope, "spec_rope", q.device, stream, (q_out, k_out), ctypes.byref(a))
    return q_out, k_out


def _sized(name, a, dev, workspace):
    """(call, workspace, its bytes) of a call that needs one; refused arguments raise."""
    L, ref = lib(), ctypes.byref(a)
    call = getattr(L, name)
    need = _on(dev, getattr(L, name + "_workspace"), ref)
    if need == 0:
        _check(call(ref, None, 0, None, None), name)
    return call, _workspace(need, dev, workspace), need


def _prompt_rows(q, k, row_start):
    """What prompt attention and key weights ask of q, k and row_start alike."""
    torch = _torch()
    if not isinstance(q, torch.Tensor):
        raise TypeError("q must be a torch.Tensor")
    dev = q.device
    q_ptr, rows, Hq, d, q_step = _rows(q, "q", q.dtype, dev)
    k_ptr, k_rows, Hkv, k_d, k_step = _rows(k, "k", q.dtype, dev)
    start = _fast(row_start, "row_start", torch.int32, dev, dev.index)
    if q.dim() != 3 or k.dim() != 3 or k_rows != rows or k_d != d:
        raise ValueError("q must be [n_rows][Hq][d], k and v [n_rows][Hkv][d]")
    return dev, _dtype_code(q), row_start.numel() - 1, (rows, Hq, Hkv, d), (q_ptr, k_ptr, start), (q_step, k_step)


def prompt_attn_args(q, k, v, row_start, out=None, lse=None, scale=0.0):
    """Build the C argument struct for prompt_attention (tensors are validated here); returns (args, out, lse)."""
    torch = _torch()
    dev, code, B, (rows, Hq, Hkv, d), (q_ptr, k_ptr, start), (q_step, k_step) = _prompt_rows(q, k, row_start)
    v_ptr, v_rows, v_heads, v_d, v_step = _rows(v, "v", q.dtype, dev)
    if v.dim() != 3 or (v_rows, v_heads, v_d) != (rows, Hkv, d):
        raise ValueError("q must be [n_rows][Hq][d], k and v [n_rows][Hkv][d]")
    if out is None:
        out = torch.empty((rows, Hq, d), dtype=q.dtype, device=dev)
    if lse is None:
        lse = torch.empty((rows, Hq), dtype=torch.float32, device=dev)
    ptr = _fast(out, "out", q.dtype, dev, dev.index), _fast(lse, "lse", torch.float32, dev, dev.index)
    if out.shape != (rows, Hq, d) or lse.shape != (rows, Hq):
        raise ValueError("out must be [n_rows][Hq][d], lse [n_rows][Hq]")
    a = PromptAttnArgs(code, B, Hq, Hkv, d, float(scale), rows, q_step, k_step, v_step, q_ptr, k_ptr, v_ptr, start, *ptr)
    return a, out, lse


def prompt_attention(q, k, v, row_start, out=None, lse=None, scale=0.0, workspace=None, dev_status=None, stream=None):
    """Causal attention over packed prompts (see spec_prompt_attention): q [n_rows][Hq][d], k and v [n_rows][Hkv][d] in
    bf16, views of wider rows included, request b's rows at ``row_start[b]`` up to ``row_start[b + 1]``.  Returns (out, lse)."""
    if stream is None and workspace is None:
        r = _native().prompt_attend(q, k, v, row_start, out, lse, scale, dev_status)
        if r is not None:
            return _answer(r, "spec_prompt_attention")
    a, out, lse = prompt_attn_args(q, k, v, row_start, out, lse, scale)
    dev = q.device
    call, ws, need = _sized("spec_prompt_attention", a, dev, workspace)
    _launch(call, "spec_prompt_attention", dev, stream, (ws, out, lse), ctypes.byref(a), ws.data_ptr(), need,
            _status_ptr(dev_status, dev))
    return out, lse


def key_weights_args(q, k, lse, row_start, window, weight=None, scale=0.0):
    """Build the C argument struct for prompt_key_weights (tensors are validated here); returns (args, weight)."""
    torch = _torch()
    dev, code, B, (rows, Hq, Hkv, d), (q_ptr, k_ptr, start), (q_step, k_step) = _prompt_rows(q, k, row_start)
    lse_ptr = _fast(lse, "lse", torch.float32, dev, dev.index)
    if weight is None:
        weight = torch.empty((Hkv, rows), dtype=torch.float32, device=dev)
    ptr = _fast(weight, "weight", torch.float32, dev, dev.index)
    if lse.shape != (rows, Hq) or weight.shape != (Hkv, rows):
        raise ValueError("lse must be [n_rows][Hq], weight [Hkv][n_rows]")
    a = KeyWeightsArgs(code, B, Hq, Hkv, d, float(scale), _clip(window), 0, rows, q_step, k_step, q_ptr, k_ptr, lse_ptr, start, ptr)
    return a, weight


def prompt_key_weights(q, k, lse, row_start, window, weight=None, scale=0.0, workspace=None, dev_status=None, stream=None):
    """The attention weight that each key gets from the last ``window`` rows of its prompt, summed over them and over the
    heads that share it (see spec_prompt_key_weights); ``lse`` is prompt_attention's.  Returns weight [Hkv][n_rows]."""
    if stream is None and workspace is None:
        r = _native().key_weights(q, k, lse, row_start, window, weight, scale, dev_status)
        if r is not None:
            return _answer(r, "spec_prompt_key_weights")
    a, weight = key_weights_args(q, k, lse, row_start, window, weight, scale)
    dev = q.device
    call, ws, need = _sized("spec_prompt_key_weights", a, dev, workspace)
    _launch(call, "spec_prompt_key_weights", dev, stream, (ws, weight), ctypes.byref(a), ws.data_ptr(), need,
            _status_ptr(dev_status, dev))
    return weight


def kv_keep_args(k, v, weight, row_start, budget, first=0, last=0, rows_out=None, outputs=None):
    """Build the C argument struct for kv_keep (tensors are validated here); returns (args, outputs), the outputs being
    (k_out, v_out, index, keep_start, n_keep)."""
    torch = _torch()
    if not isinstance(k, torch.Tensor):
        raise TypeError("k must be a torch.Tensor")
    dev, dtype, i32 = k.device, k.dtype, torch.int32
    ix, code = dev.index, _dtype_code(k)
    k_ptr, rows, Hkv, d, k_step = _rows(k, "k", dtype, dev)
    v_ptr, _, _, _, v_step = _rows(v, "v", dtype, dev)
    if k.dim() != 3 or v.shape != k.shape:
        raise ValueError("k and v must be [n_rows][Hkv][d]")
    w_ptr = _fast(weight, "weight", torch.float32, dev, ix)
    start = _fast(row_start, "row_start", i32, dev, ix)
    if weight.shape != (Hkv, rows):
        raise ValueError("weight must be [Hkv][n_rows]")
    B = row_start.numel() - 1
    if outputs is None:
        n_out = max(0, min(rows, B * _clip(budget))) if rows_out is None else int(rows_out)
        outputs = (torch.empty((n_out, Hkv, d), dtype=dtype, device=dev), torch.empty((n_out, Hkv, d), dtype=dtype, device=dev),
                   torch.empty((n_out, Hkv), dtype=i32, device=dev), torch.empty(B + 1, dtype=i32, device=dev),
                   torch.empty(B, dtype=i32, device=dev))
    k_out, v_out, index, keep_start, n_keep = outputs
    ptr = (_fast(k_out, "k_out", dtype, dev, ix), _fast(v_out, "v_out", dtype, dev, ix), _fast(index, "index", i32, dev, ix),
           _fast(keep_start, "keep_start", i32, dev, ix), _fast(n_keep, "n_keep", i32, dev, ix))
    n_out = k_out.shape[0]
    if k_out.shape != (n_out, Hkv, d) or v_out.shape != k_out.shape or index.shape != (n_out, Hkv) or \
            keep_start.numel() != B + 1 or n_keep.numel() != B:
        raise ValueError("k_out and v_out must be [rows_out][Hkv][d], index [rows_out][Hkv], keep_start [B + 1], n_keep [B]")
    if rows_out is not None and int(rows_out) != n_out:
        raise ValueError("rows_out is the number of rows of the outputs")
    a = KvKeepArgs(code, B, Hkv, d, _clip(budget), _clip(first), _clip(last), 0, rows, n_out, k_step, v_step, k_ptr, v_ptr, w_ptr,
                   start, *ptr)
    return a, outputs


def kv_keep(k, v, weight, row_start, budget, first=0, last=0, rows_out=None, outputs=None, workspace=None, dev_status=None,
            stream=None):
    """The rows of each prompt that ``budget`` leaves, per KV head: its first ``first`` and last ``last`` rows and those with
    the largest weights, in the prompt's order (see spec_kv_keep).  ``rows_out`` bounds the rows kept in all (default: the
    rows there are, or the budgets' sum; the rows of ``outputs`` where these are given).  Returns (k_out, v_out, index, keep_start, n_keep); keep_start and n_keep are the
    row_start and n_new with which kv_reserve and kv8_append admit the rows."""
    if stream is None and workspace is None:
        r = _native().keep(k, v, weight, row_start, budget, first, last, rows_out, outputs, dev_status)
        if r is not None:
            return _answer(r, "spec_kv_keep")
    a, outputs = kv_keep_args(k, v, weight, row_start, budget, first, last, rows_out, outputs)
    dev = k.device
    call, ws, need = _sized("spec_kv_keep", a, dev, workspace)
    _launch(call, "spec_kv_keep", dev, stream, (ws,) + tuple(outputs), ctypes.byref(a), ws.data_ptr(), need,
            _status_ptr(dev_status, dev))
    return outputs
