// The 8-bit cache's calls for Python, without the interpreter's share: checks of the tensors, new outputs and the C
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

// A call's arguments.  The first thing that is not plain clears `ok`; nothing is read from a tensor after that.
struct Call {
  bool ok = true;
  int device = -1;  // of the first tensor

  const Tensor* tensor(PyObject* o, at::ScalarType type) {
    if (!ok || !THPVariable_CheckExact(o)) return fail();
    const Tensor& t = THPVariable_Unpack(o);
    if (t.scalar_type() != type || !t.is_cuda() || !t.is_contiguous()) return fail();
    const int at = t.device().index();
    if (device < 0) {
      device = at;
      if (c10::cuda::current_device() != at) return fail();
    } else if (device != at) {
      return fail();
    }
    return &t;
  }
  const Tensor* ints(PyObject* o, int64_t count) {  // int32 of `count` elements (any number: -1)
    const Tensor* t = tensor(o, at::kInt);
    return t && (count < 0 || t->numel() == count) ? t : fail();
  }
  const Tensor* shaped(PyObject* o, at::ScalarType type, c10::IntArrayRef shape) {
    const Tensor* t = tensor(o, type);
    return t && t->sizes() == shape ? t : fail();
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

PyMethodDef methods[] = {{"bind", (PyCFunction)(void*)bind, METH_FASTCALL, nullptr},
                         {"reserve", (PyCFunction)(void*)reserve, METH_FASTCALL, nullptr},
                         {"append", (PyCFunction)(void*)append, METH_FASTCALL, nullptr},
                         {"attend", (PyCFunction)(void*)attend, METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "spectree_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" PyObject* PyInit_spectree_marshal() { return PyModule_Create(&module); }
