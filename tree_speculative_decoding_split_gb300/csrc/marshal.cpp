// The 8-bit cache's and the prompts' calls for Python, without the interpreter's share: checks of the tensors, new outputs and the C
// call.  These calls come once per layer and token, where 15 to 27 us of attribute look-ups were more than the
// kernels.  Every function answers for the plain call only (tensors as documented, on the current device and its
// current stream) and returns None for any other, which the binding's own checks then carry out or refuse; a number is
// the C call's error.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "spectree.h"

namespace {

using at::Tensor;

// Addresses of the C entry points, handed over by the binding (which has the library open).
using ReserveFn = spec_status (*)(const spec_kv_reserve_args*, int32_t*, void*);
using AppendFn = spec_status (*)(const spec_kv8_append_args*, int32_t*, void*);
using WorkspaceFn = size_t (*)(const spec_attn_kv8_args*);
using AttendFn = spec_status (*)(const spec_attn_kv8_args*, void*, size_t, int32_t*, void*);
ReserveFn g_reserve = nullptr;
AppendFn g_append = nullptr;
WorkspaceFn g_workspace = nullptr;
AttendFn g_attend = nullptr;
using PositionsFn = spec_status (*)(const spec_rope_positions_args*, int32_t*, void*);
using RopeFn = spec_status (*)(const spec_rope_args*, void*);
template <typename Args>
struct Sized {  // a call with a workspace
  size_t (*size)(const Args*) = nullptr;
  spec_status (*call)(const Args*, void*, size_t, int32_t*, void*) = nullptr;
};
PositionsFn g_positions = nullptr;
RopeFn g_rope = nullptr;
Sized<spec_prompt_attn_args> g_prompt;
Sized<spec_key_weights_args> g_weights;
Sized<spec_kv_keep_args> g_keep;

// A call's arguments.  The first thing that is not plain clears `ok`; nothing is read from a tensor after that.
struct Call {
  bool ok = true;
  int device = -1;  // of the first tensor

  const Tensor* tensor(PyObject* o, at::ScalarType type) {
    if (!ok || !THPVariable_CheckExact(o)) return fail();
    const Tensor& t = THPVariable_Unpack(o);
    if (t.scalar_type() != type || !t.is_cuda() || !t.is_contiguous()) return fail();
    return same_device(t) ? &t : fail();
  }
  const Tensor* ints(PyObject* o, int64_t count) {  // int32 of `count` elements (any number: -1)
    const Tensor* t = tensor(o, at::kInt);
    return t && (count < 0 || t->numel() == count) ? t : fail();
  }
  const Tensor* shaped(PyObject* o, at::ScalarType type, c10::IntArrayRef shape) {
    const Tensor* t = tensor(o, type);
    return t && t->sizes() == shape ? t : fail();
  }
  // Rows of heads [rows][H][d], or [B][N][H][d] where `batched` allows it: the heads of a row together, the rows at one
  // distance (*step elements), as in a view of wider rows.
  const Tensor* rows(PyObject* o, at::ScalarType type, int64_t* step, bool batched = false) {
    if (!ok || !THPVariable_CheckExact(o)) return fail();
    const Tensor& t = THPVariable_Unpack(o);
    const int64_t dim = t.dim();
    if (t.scalar_type() != type || !t.is_cuda() || (dim != 3 && !(batched && dim == 4)) || t.numel() == 0) return fail();
    const auto size = t.sizes(), stride = t.strides();
    const int64_t H = size[dim - 2], d = size[dim - 1];
    if (stride[dim - 1] != 1 || (H > 1 && stride[dim - 2] != d)) return fail();
    *step = size[dim - 3] > 1 ? stride[dim - 3] : H * d;
    if (dim == 4 && size[0] > 1) {
      if (size[1] == 1)
        *step = stride[0];
      else if (stride[0] != size[1] * stride[1])
        return fail();
    }
    return same_device(t) ? &t : fail();
  }
  float number(PyObject* o) {
    if (!PyFloat_CheckExact(o)) {
      ok = false;
      return 0.f;
    }
    return (float)PyFloat_AS_DOUBLE(o);
  }
  int64_t integer(PyObject* o) {
    if (!PyLong_CheckExact(o)) {
      ok = false;
      return 0;
    }
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
      PyErr_Clear();
      ok = false;
    }
    return v;
  }
  int32_t* status(PyObject* o) {  // dev_status or None
    if (o == Py_None) return nullptr;
    const Tensor* t = tensor(o, at::kInt);
    return t ? static_cast<int32_t*>(t->data_ptr()) : nullptr;
  }
  Tensor make(c10::IntArrayRef shape, at::ScalarType type) const {
    return at::empty(shape, at::TensorOptions().dtype(type).device(at::kCUDA, (c10::DeviceIndex)device));
  }
  void* stream() const { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream(); }

 private:
  bool same_device(const Tensor& t) {
    const int at = t.device().index();
    if (device < 0) {
      device = at;
      return c10::cuda::current_device() == at;
    }
    return device == at;
  }
  const Tensor* fail() {
    ok = false;
    return nullptr;
  }
};

template <typename T>
T* ptr(const Tensor* t) {
  return static_cast<T*>(t->data_ptr());
}
template <typename T>
T* ptr(const Tensor& t) {
  return static_cast<T*>(t.data_ptr());
}

// The pools, scales and table: k_cache, v_cache, k_scale, v_scale, table (o[0 .. 4]).
struct Pools {
  const Tensor *k, *v, *ks, *vs, *table;
  int64_t blocks, heads, bs, d, max_blocks;
};
bool pools(Call& c, PyObject* const* o, int64_t batch, Pools* p) {
  p->k = c.tensor(o[0], at::kFloat8_e4m3fn);
  if (!p->k || p->k->dim() != 4) return false;
  p->v = c.shaped(o[1], at::kFloat8_e4m3fn, p->k->sizes());
  p->ks = c.shaped(o[2], at::kFloat, p->k->sizes().slice(0, 2));
  p->vs = c.shaped(o[3], at::kFloat, p->k->sizes().slice(0, 2));
  p->table = c.ints(o[4], -1);
  if (!c.ok || p->table->dim() != 2 || p->table->size(0) != batch) return false;
  p->blocks = p->k->size(0);
  p->heads = p->k->size(1);
  p->bs = p->k->size(2);
  p->d = p->k->size(3);
  p->max_blocks = p->table->size(1);
  return true;
}

bool fits(std::initializer_list<int64_t> sizes) {
  for (const int64_t s : sizes)
    if (s < 0 || s > INT32_MAX) return false;
  return true;
}

// Runs `body`, which returns a new reference, or null for a call that is not plain; C++ exceptions become Python's.
template <typename F>
PyObject* guarded(F&& body) {
  HANDLE_TH_ERRORS
  PyObject* r = body();
  if (r || PyErr_Occurred()) return r;
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

PyObject* pair(PyObject* a, PyObject* b) {  // takes both references
  PyObject* t = a && b ? PyTuple_Pack(2, a, b) : nullptr;
  Py_XDECREF(a);
  Py_XDECREF(b);
  return t;
}
PyObject* same(PyObject* o) {
  Py_INCREF(o);
  return o;
}

PyObject* bind(PyObject*, PyObject* const* o, Py_ssize_t n) {
  if (n != 4) {
    PyErr_SetString(PyExc_TypeError, "four addresses");
    return nullptr;
  }
  void* at[4];
  for (int i = 0; i < 4; ++i) at[i] = PyLong_AsVoidPtr(o[i]);
  if (PyErr_Occurred()) return nullptr;
  g_reserve = reinterpret_cast<ReserveFn>(at[0]);
  g_append = reinterpret_cast<AppendFn>(at[1]);
  g_workspace = reinterpret_cast<WorkspaceFn>(at[2]);
  g_attend = reinterpret_cast<AttendFn>(at[3]);
  Py_RETURN_NONE;
}

// seq_len, n_new, table, n_blocks, free_list, free_count, block_size, slot_cap, slot_map, row_start, dev_status
PyObject* reserve(PyObject*, PyObject* const* o, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Call c;
    if (n != 11 || !g_reserve) return nullptr;
    const Tensor* table = c.ints(o[2], -1);
    if (!table || table->dim() != 2) return nullptr;
    const int64_t B = table->size(0);
    const Tensor *len = c.ints(o[0], B), *add = c.ints(o[1], B), *held = c.ints(o[3], B), *list = c.ints(o[4], -1),
                 *count = c.ints(o[5], 1);
    const int64_t bs = c.integer(o[6]);
    const int64_t cap = o[7] == Py_None ? 0 : c.integer(o[7]);
    int32_t* status = c.status(o[10]);
    if (!c.ok || cap < 0 || !fits({B, bs, table->size(1), list->numel(), cap})) return nullptr;
    const Tensor* map = o[8] == Py_None ? nullptr : c.tensor(o[8], at::kLong);
    const Tensor* start = o[9] == Py_None ? nullptr : c.ints(o[9], B + 1);
    if (!c.ok) return nullptr;
    Tensor new_map, new_start;
    if (!map && o[7] != Py_None) {
      new_map = c.make({cap}, at::kLong);
      map = &new_map;
    }
    if (!start) {
      new_start = c.make({B + 1}, at::kInt);
      start = &new_start;
    }
    spec_kv_reserve_args a = {};
    a.batch = (int32_t)B;
    a.block_size = (int32_t)bs;
    a.max_blocks = (int32_t)table->size(1);
    a.num_blocks = (int32_t)list->numel();
    a.slot_cap = map ? map->numel() : 0;
    a.seq_len = ptr<int32_t>(len);
    a.n_new = ptr<int32_t>(add);
    a.block_table = ptr<int32_t>(table);
    a.n_blocks = ptr<int32_t>(held);
    a.free_list = ptr<int32_t>(list);
    a.free_count = ptr<int32_t>(count);
    if (map && a.slot_cap > 0) a.slot_map = ptr<int64_t>(map);
    // an empty tensor has no address; any other says that there is a map, and nothing is written to it
    if (map && a.slot_cap == 0) a.slot_map = reinterpret_cast<int64_t*>(ptr<int32_t>(start));
    a.row_start = ptr<int32_t>(start);
    const spec_status st = g_reserve(&a, status, c.stream());
    if (st != SPEC_OK) return PyLong_FromLong(st);
    return pair(new_map.defined() ? THPVariable_Wrap(new_map) : same(o[8]),
                new_start.defined() ? THPVariable_Wrap(new_start) : same(o[9]));
  });
}

// k_new, v_new, k_cache, v_cache, k_scale, v_scale, table, seq_len, row_start, path, accept_len, new_len, dev_status
PyObject* append(PyObject*, PyObject* const* o, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Call c;
    if (n != 13 || !g_append || !THPVariable_CheckExact(o[0])) return nullptr;
    const at::ScalarType type = THPVariable_Unpack(o[0]).scalar_type();
    if (type != at::kBFloat16 && type != at::kFloat) return nullptr;
    const Tensor* k = c.tensor(o[0], type);
    const Tensor* len = c.ints(o[7], -1);
    if (!c.ok || k->numel() == 0) return nullptr;
    const Tensor* v = c.shaped(o[1], type, k->sizes());
    const int64_t B = len->numel(), dim = k->dim();
    Pools p;
    if (!pools(c, o + 2, B, &p) || dim < 3 || k->size(dim - 2) != p.heads || k->size(dim - 1) != p.d) return nullptr;
    spec_kv8_append_args a = {};
    if (o[9] != Py_None) {
      const Tensor *path = c.ints(o[9], -1), *accept = c.ints(o[10], B);
      if (!c.ok || o[8] != Py_None || dim != 4 || k->size(0) != B || path->dim() != 2 || path->size(0) != B) return nullptr;
      if (!fits({k->size(1), path->size(1)})) return nullptr;
      a.n_max = (int32_t)k->size(1);
      a.path_cap = (int32_t)path->size(1);
      a.path = ptr<int32_t>(path);
      a.accept_len = ptr<int32_t>(accept);
    } else {
      const Tensor* start = c.ints(o[8], B + 1);
      if (!c.ok || o[10] != Py_None || dim != 3) return nullptr;
      a.n_rows = k->size(0);
      a.row_start = ptr<int32_t>(start);
    }
    const Tensor* new_len = o[11] == Py_None ? nullptr : c.ints(o[11], B);
    int32_t* status = c.status(o[12]);
    if (!c.ok || !fits({B, p.heads, p.d, p.bs, p.max_blocks, p.blocks})) return nullptr;
    Tensor made;
    if (!new_len) {
      made = c.make({B}, at::kInt);
      new_len = &made;
    }
    a.dtype = type == at::kBFloat16 ? SPEC_DTYPE_BF16 : SPEC_DTYPE_F32;
    a.batch = (int32_t)B;
    a.num_kv_heads = (int32_t)p.heads;
    a.head_dim = (int32_t)p.d;
    a.block_size = (int32_t)p.bs;
    a.max_blocks = (int32_t)p.max_blocks;
    a.num_blocks = (int32_t)p.blocks;
    a.k_new = k->data_ptr();
    a.v_new = v->data_ptr();
    a.seq_len = ptr<int32_t>(len);
    a.block_table = ptr<int32_t>(p.table);
    a.k_cache = ptr<uint8_t>(p.k);
    a.v_cache = ptr<uint8_t>(p.v);
    a.k_scale = ptr<float>(p.ks);
    a.v_scale = ptr<float>(p.vs);
    a.new_len = ptr<int32_t>(new_len);
    const spec_status st = g_append(&a, status, c.stream());
    if (st != SPEC_OK) return PyLong_FromLong(st);
    return made.defined() ? THPVariable_Wrap(made) : same(o[11]);
  });
}

// q, k_tree, v_tree, k_cache, v_cache, k_scale, v_scale, table, prefix_len, n_nodes, parent, out, lse, scale, dev_status
PyObject* attend(PyObject*, PyObject* const* o, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Call c;
    if (n != 15 || !g_attend) return nullptr;
    const Tensor* q = c.tensor(o[0], at::kBFloat16);
    if (!q || q->dim() != 4 || !PyFloat_CheckExact(o[13])) return nullptr;
    const int64_t B = q->size(0), N = q->size(1), Hq = q->size(2), d = q->size(3);
    Pools p;
    if (!pools(c, o + 3, B, &p) || p.d != d) return nullptr;
    const Tensor* kt = c.shaped(o[1], at::kBFloat16, {B, N, p.heads, d});
    const Tensor* vt = c.shaped(o[2], at::kBFloat16, {B, N, p.heads, d});
    const Tensor *len = c.ints(o[8], B), *nodes = c.ints(o[9], B), *parent = c.shaped(o[10], at::kInt, {B, N});
    const Tensor* out = o[11] == Py_None ? nullptr : c.shaped(o[11], at::kBFloat16, q->sizes());
    const Tensor* lse = o[12] == Py_None ? nullptr : c.shaped(o[12], at::kFloat, {B, N, Hq});
    int32_t* status = c.status(o[14]);
    if (!c.ok || !fits({B, N, Hq, p.heads, d, p.bs, p.max_blocks, p.blocks})) return nullptr;
    spec_attn_kv8_args a = {};
    a.dtype = SPEC_DTYPE_BF16;
    a.batch = (int32_t)B;
    a.n_max = (int32_t)N;
    a.num_q_heads = (int32_t)Hq;
    a.num_kv_heads = (int32_t)p.heads;
    a.head_dim = (int32_t)d;
    a.block_size = (int32_t)p.bs;
    a.max_blocks = (int32_t)p.max_blocks;
    a.num_blocks = (int32_t)p.blocks;
    a.scale = (float)PyFloat_AS_DOUBLE(o[13]);
    a.q = q->data_ptr();
    a.k_tree = kt->data_ptr();
    a.v_tree = vt->data_ptr();
    a.k_cache = ptr<uint8_t>(p.k);
    a.v_cache = ptr<uint8_t>(p.v);
    a.k_scale = ptr<float>(p.ks);
    a.v_scale = ptr<float>(p.vs);
    a.prefix_len = ptr<int32_t>(len);
    a.n_nodes = ptr<int32_t>(nodes);
    a.parent = ptr<int32_t>(parent);
    a.block_table = ptr<int32_t>(p.table);
    Tensor new_out, new_lse;
    if (!out) {
      new_out = c.make(q->sizes(), at::kBFloat16);
      out = &new_out;
    }
    if (!lse) {
      new_lse = c.make({B, N, Hq}, at::kFloat);
      lse = &new_lse;
    }
    a.out = out->data_ptr();
    a.lse = ptr<float>(lse);
    const size_t need = g_workspace(&a);
    if (need == 0) return nullptr;  // refused: the binding asks again and says why
    const Tensor ws = c.make({(int64_t)need}, at::kByte);
    const spec_status st = g_attend(&a, ws.data_ptr(), need, status, c.stream());
    if (st != SPEC_OK) return PyLong_FromLong(st);
    return pair(new_out.defined() ? THPVariable_Wrap(new_out) : same(o[11]),
                new_lse.defined() ? THPVariable_Wrap(new_lse) : same(o[12]));
  });
}

PyObject* bind_prompt(PyObject*, PyObject* const* o, Py_ssize_t n) {
  if (n != 8) {
    PyErr_SetString(PyExc_TypeError, "eight addresses");
    return nullptr;
  }
  void* at[8];
  for (int i = 0; i < 8; ++i) at[i] = PyLong_AsVoidPtr(o[i]);
  if (PyErr_Occurred()) return nullptr;
  g_positions = reinterpret_cast<PositionsFn>(at[0]);
  g_rope = reinterpret_cast<RopeFn>(at[1]);
  g_prompt.size = reinterpret_cast<decltype(g_prompt.size)>(at[2]);
  g_prompt.call = reinterpret_cast<decltype(g_prompt.call)>(at[3]);
  g_weights.size = reinterpret_cast<decltype(g_weights.size)>(at[4]);
  g_weights.call = reinterpret_cast<decltype(g_weights.call)>(at[5]);
  g_keep.size = reinterpret_cast<decltype(g_keep.size)>(at[6]);
  g_keep.call = reinterpret_cast<decltype(g_keep.call)>(at[7]);
  Py_RETURN_NONE;
}

// The call with a workspace of its own; -1 where it is refused (the binding asks again and says why).
template <typename Args>
int with_workspace(const Sized<Args>& f, const Args& a, const Call& c, int32_t* status) {
  const size_t need = f.size(&a);
  if (need == 0) return -1;
  const Tensor ws = c.make({(int64_t)need}, at::kByte);
  return f.call(&a, ws.data_ptr(), need, status, c.stream());
}

// pos0, row_start, n_rows, parent, n_nodes, positions, dev_status
PyObject* positions(PyObject*, PyObject* const* o, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Call c;
    if (n != 7 || !g_positions || (o[1] == Py_None) == (o[3] == Py_None)) return nullptr;
    const Tensor* pos0 = c.ints(o[0], -1);
    if (!pos0) return nullptr;
    const int64_t B = pos0->numel();
    const bool trees = o[3] != Py_None;
    spec_rope_positions_args a = {};
    Tensor made;
    const Tensor* out = nullptr;
    if (trees) {
      const Tensor *parent = c.ints(o[3], -1), *nodes = c.ints(o[4], B);
      if (!c.ok || o[2] != Py_None || parent->dim() != 2 || parent->size(0) != B || !fits({parent->size(1)})) return nullptr;
      a.n_max = (int32_t)parent->size(1);
      a.parent = ptr<int32_t>(parent);
      a.n_nodes = ptr<int32_t>(nodes);
      out = o[5] == Py_None ? nullptr : c.shaped(o[5], at::kInt, parent->sizes());
      if (c.ok && !out) out = &(made = c.make(parent->sizes(), at::kInt));
    } else {
      const Tensor* start = c.ints(o[1], B + 1);
      if (!c.ok || o[4] != Py_None || o[2] == Py_None) return nullptr;
      a.n_rows = c.integer(o[2]);
      if (!c.ok || a.n_rows < 1) return nullptr;
      a.row_start = ptr<int32_t>(start);
      out = o[5] == Py_None ? nullptr : c.shaped(o[5], at::kInt, {a.n_rows});
      if (c.ok && !out) out = &(made = c.make({a.n_rows}, at::kInt));
      a.fill = made.defined();
    }
    int32_t* status = c.status(o[6]);
    if (!c.ok || !fits({B})) return nullptr;
    a.batch = (int32_t)B;
    a.pos0 = ptr<int32_t>(pos0);
    a.positions = ptr<int32_t>(out);
    const spec_status st = g_positions(&a, status, c.stream());
    if (st != SPEC_OK) return PyLong_FromLong(st);
    return made.defined() ? THPVariable_Wrap(made) : same(o[5]);
  });
}

// q, k, positions, turns, layout, amplitude, q_out, k_out
PyObject* rope(PyObject*, PyObject* const* o, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Call c;
    if (n != 8 || !g_rope || !THPVariable_CheckExact(o[0])) return nullptr;
    const at::ScalarType type = THPVariable_Unpack(o[0]).scalar_type();
    if (type != at::kBFloat16 && type != at::kFloat) return nullptr;
    spec_rope_args a = {};
    const Tensor *q = c.rows(o[0], type, &a.q_stride, true), *k = c.rows(o[1], type, &a.k_stride, true);
    const Tensor* turns = c.tensor(o[3], at::kLong);
    if (!c.ok) return nullptr;
    const int64_t dim = q->dim(), Hq = q->size(dim - 2), d = q->size(dim - 1), Hk = k->size(k->dim() - 2);
    a.n_rows = q->numel() / (Hq * d);
    const Tensor* pos = c.ints(o[2], a.n_rows);
    if (!c.ok || k->size(k->dim() - 1) != d || k->numel() != a.n_rows * Hk * d || !fits({Hq, Hk, d, 2 * turns->numel()}))
      return nullptr;
    const int64_t layout = c.integer(o[4]);
    a.amplitude = c.number(o[5]);
    const Tensor* qo = o[6] == Py_None ? nullptr : c.rows(o[6], type, &a.q_out_stride, true);
    const Tensor* ko = o[7] == Py_None ? nullptr : c.rows(o[7], type, &a.k_out_stride, true);
    if (!c.ok || (qo && qo->sizes() != q->sizes()) || (ko && ko->sizes() != k->sizes())) return nullptr;
    Tensor q_made, k_made;
    if (!qo) {
      qo = &(q_made = c.make(q->sizes(), type));
      a.q_out_stride = Hq * d;
    }
    if (!ko) {
      ko = &(k_made = c.make(k->sizes(), type));
      a.k_out_stride = Hk * d;
    }
    a.dtype = type == at::kBFloat16 ? SPEC_DTYPE_BF16 : SPEC_DTYPE_F32;
    a.layout = (int32_t)layout;
    a.num_q_heads = (int32_t)Hq;
    a.num_k_heads = (int32_t)Hk;
    a.head_dim = (int32_t)d;
    a.rot_dim = (int32_t)(2 * turns->numel());
    a.q = q->data_ptr();
    a.k = k->data_ptr();
    a.positions = ptr<int32_t>(pos);
    a.turns = ptr<int64_t>(turns);
    a.q_out = qo->data_ptr();
    a.k_out = ko->data_ptr();
    const spec_status st = g_rope(&a, c.stream());
    if (st != SPEC_OK) return PyLong_FromLong(st);
    return pair(q_made.defined() ? THPVariable_Wrap(q_made) : same(o[6]), k_made.defined() ? THPVariable_Wrap(k_made) : same(o[7]));
  });
}

// q, k, v, row_start, out, lse, scale, dev_status
PyObject* prompt_attend(PyObject*, PyObject* const* o, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Call c;
    if (n != 8 || !g_prompt.call) return nullptr;
    spec_prompt_attn_args a = {};
    const Tensor *q = c.rows(o[0], at::kBFloat16, &a.q_stride), *k = c.rows(o[1], at::kBFloat16, &a.k_stride);
    const Tensor *v = c.rows(o[2], at::kBFloat16, &a.v_stride), *start = c.ints(o[3], -1);
    if (!c.ok || k->size(0) != q->size(0) || k->size(2) != q->size(2) || v->sizes() != k->sizes()) return nullptr;
    const int64_t rows = q->size(0), Hq = q->size(1), Hkv = k->size(1), d = q->size(2), B = start->numel() - 1;
    const Tensor* out = o[4] == Py_None ? nullptr : c.shaped(o[4], at::kBFloat16, q->sizes());
    const Tensor* lse = o[5] == Py_None ? nullptr : c.shaped(o[5], at::kFloat, {rows, Hq});
    a.scale = c.number(o[6]);
    int32_t* status = c.status(o[7]);
    if (!c.ok || !fits({Hq, Hkv, d, B})) return nullptr;
    Tensor out_made, lse_made;
    if (!out) out = &(out_made = c.make(q->sizes(), at::kBFloat16));
    if (!lse) lse = &(lse_made = c.make({rows, Hq}, at::kFloat));
    a.dtype = SPEC_DTYPE_BF16;
    a.batch = (int32_t)B;
    a.num_q_heads = (int32_t)Hq;
    a.num_kv_heads = (int32_t)Hkv;
    a.head_dim = (int32_t)d;
    a.n_rows = rows;
    a.q = q->data_ptr();
    a.k = k->data_ptr();
    a.v = v->data_ptr();
    a.row_start = ptr<int32_t>(start);
    a.out = out->data_ptr();
    a.lse = ptr<float>(lse);
    const int st = with_workspace(g_prompt, a, c, status);
    if (st < 0) return nullptr;
    if (st != SPEC_OK) return PyLong_FromLong(st);
    return pair(out_made.defined() ? THPVariable_Wrap(out_made) : same(o[4]),
                lse_made.defined() ? THPVariable_Wrap(lse_made) : same(o[5]));
  });
}

// q, k, lse, row_start, window, weight, scale, dev_status
PyObject* key_weights(PyObject*, PyObject* const* o, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Call c;
    if (n != 8 || !g_weights.call) return nullptr;
    spec_key_weights_args a = {};
    const Tensor *q = c.rows(o[0], at::kBFloat16, &a.q_stride), *k = c.rows(o[1], at::kBFloat16, &a.k_stride);
    if (!c.ok || k->size(0) != q->size(0) || k->size(2) != q->size(2)) return nullptr;
    const int64_t rows = q->size(0), Hq = q->size(1), Hkv = k->size(1), d = q->size(2);
    const Tensor *lse = c.shaped(o[2], at::kFloat, {rows, Hq}), *start = c.ints(o[3], -1);
    const int64_t window = c.integer(o[4]);
    const Tensor* weight = o[5] == Py_None ? nullptr : c.shaped(o[5], at::kFloat, {Hkv, rows});
    a.scale = c.number(o[6]);
    int32_t* status = c.status(o[7]);
    if (!c.ok || !fits({Hq, Hkv, d, window, start->numel() - 1})) return nullptr;
    Tensor made;
    if (!weight) weight = &(made = c.make({Hkv, rows}, at::kFloat));
    a.dtype = SPEC_DTYPE_BF16;
    a.batch = (int32_t)(start->numel() - 1);
    a.num_q_heads = (int32_t)Hq;
    a.num_kv_heads = (int32_t)Hkv;
    a.head_dim = (int32_t)d;
    a.window = (int32_t)window;
    a.n_rows = rows;
    a.q = q->data_ptr();
    a.k = k->data_ptr();
    a.lse = ptr<float>(lse);
    a.row_start = ptr<int32_t>(start);
    a.weight = ptr<float>(weight);
    const int st = with_workspace(g_weights, a, c, status);
    if (st < 0) return nullptr;
    if (st != SPEC_OK) return PyLong_FromLong(st);
    return made.defined() ? THPVariable_Wrap(made) : same(o[5]);
  });
}

// k, v, weight, row_start, budget, first, last, rows_out, outputs, dev_status
PyObject* keep(PyObject*, PyObject* const* o, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Call c;
    if (n != 10 || !g_keep.call || o[8] != Py_None || !THPVariable_CheckExact(o[0])) return nullptr;
    const at::ScalarType type = THPVariable_Unpack(o[0]).scalar_type();
    if (type != at::kBFloat16 && type != at::kFloat) return nullptr;
    spec_kv_keep_args a = {};
    const Tensor *k = c.rows(o[0], type, &a.k_stride), *v = c.rows(o[1], type, &a.v_stride);
    if (!c.ok || v->sizes() != k->sizes()) return nullptr;
    const int64_t rows = k->size(0), Hkv = k->size(1), d = k->size(2);
    const Tensor *weight = c.shaped(o[2], at::kFloat, {Hkv, rows}), *start = c.ints(o[3], -1);
    const int64_t budget = c.integer(o[4]), first = c.integer(o[5]), last = c.integer(o[6]);
    if (!c.ok) return nullptr;
    const int64_t B = start->numel() - 1;
    if (!fits({Hkv, d, budget, first, last, B})) return nullptr;
    const int64_t out_rows = o[7] == Py_None ? (rows < B * budget ? rows : B * budget) : c.integer(o[7]);
    int32_t* status = c.status(o[9]);
    if (!c.ok || out_rows < 1 || B < 1) return nullptr;
    Tensor made[5] = {c.make({out_rows, Hkv, d}, type), c.make({out_rows, Hkv, d}, type), c.make({out_rows, Hkv}, at::kInt),
                      c.make({B + 1}, at::kInt), c.make({B}, at::kInt)};
    a.dtype = type == at::kBFloat16 ? SPEC_DTYPE_BF16 : SPEC_DTYPE_F32;
    a.batch = (int32_t)B;
    a.num_kv_heads = (int32_t)Hkv;
    a.head_dim = (int32_t)d;
    a.budget = (int32_t)budget;
    a.first = (int32_t)first;
    a.last = (int32_t)last;
    a.n_rows = rows;
    a.rows_out = out_rows;
    a.k = k->data_ptr();
    a.v = v->data_ptr();
    a.weight = ptr<float>(weight);
    a.row_start = ptr<int32_t>(start);
    a.k_out = made[0].data_ptr();
    a.v_out = made[1].data_ptr();
    a.index = ptr<int32_t>(made[2]);
    a.keep_start = ptr<int32_t>(made[3]);
    a.n_keep = ptr<int32_t>(made[4]);
    const int st = with_workspace(g_keep, a, c, status);
    if (st < 0) return nullptr;
    if (st != SPEC_OK) return PyLong_FromLong(st);
    PyObject* t = PyTuple_New(5);
    for (int i = 0; t && i < 5; ++i) {
      PyObject* x = THPVariable_Wrap(made[i]);
      if (!x) {
        Py_CLEAR(t);
        break;
      }
      PyTuple_SET_ITEM(t, i, x);
    }
    return t;
  });
}

PyMethodDef methods[] = {{"bind", (PyCFunction)(void*)bind, METH_FASTCALL, nullptr},
                         {"reserve", (PyCFunction)(void*)reserve, METH_FASTCALL, nullptr},
                         {"append", (PyCFunction)(void*)append, METH_FASTCALL, nullptr},
                         {"attend", (PyCFunction)(void*)attend, METH_FASTCALL, nullptr},
                         {"bind_prompt", (PyCFunction)(void*)bind_prompt, METH_FASTCALL, nullptr},
                         {"positions", (PyCFunction)(void*)positions, METH_FASTCALL, nullptr},
                         {"rope", (PyCFunction)(void*)rope, METH_FASTCALL, nullptr},
                         {"prompt_attend", (PyCFunction)(void*)prompt_attend, METH_FASTCALL, nullptr},
                         {"key_weights", (PyCFunction)(void*)key_weights, METH_FASTCALL, nullptr},
                         {"keep", (PyCFunction)(void*)keep, METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "spectree_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" PyObject* PyInit_spectree_marshal() { return PyModule_Create(&module); }
