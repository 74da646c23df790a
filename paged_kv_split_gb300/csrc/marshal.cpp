// Argument marshalling of the draft-and-verify calls for Python.
//
// A decoding loop makes these calls hundreds of times a token with tensors it
// checked long ago; through ctypes their marshalling took 14 us a call on a
// Grace core, the call itself 4. Each function here does what binding.py's
// function of the same purpose does, checks included, and returns its status;
// it returns None, having done nothing, for arguments that it does not take as
// they are, and binding.py then says what is wrong with them. Tensors throw for
// what they do not have (a 0-dim tensor's sizes, a vmapped one's address): no
// exception leaves an entry, it means None too.
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include "pd.h"

// The device whose tensors are taken; a host build of the tests has the CPU's.
#ifndef PD_MARSHAL_DEVICE
#define PD_MARSHAL_DEVICE at::kCUDA
#endif

namespace {

// Unpacks arguments in order; `ok` turns false at the first that does not fit.
struct Args {
  PyObject* const* a;
  int dev = -1;
  bool ok = true;
  // a contiguous tensor of the call's device (the first tensor's), or null
  const at::Tensor* tensor(int i) {
    if (!THPVariable_CheckExact(a[i])) {
      ok = false;
      return nullptr;
    }
    const at::Tensor& t = THPVariable_Unpack(a[i]);
    if (t.device().type() != PD_MARSHAL_DEVICE || !t.is_contiguous() || (dev >= 0 && t.get_device() != dev)) ok = false;
    if (dev < 0 && ok) dev = static_cast<int>(t.get_device());
    return ok ? &t : nullptr;
  }
  void* ptr(int i, at::ScalarType type) {
    const at::Tensor* t = tensor(i);
    if (!t || t->scalar_type() != type) {
      ok = false;
      return nullptr;
    }
    return t->data_ptr();
  }
  void* ptr(int i, at::ScalarType type, int64_t n) {  // [n]
    const at::Tensor* t = tensor(i);
    if (!t || t->scalar_type() != type || t->dim() != 1 || t->size(0) != n) {
      ok = false;
      return nullptr;
    }
    return t->data_ptr();
  }
  void* optional(int i, at::ScalarType type, int64_t n) {
    return a[i] == Py_None ? nullptr : ptr(i, type, n);
  }
  void* bytes(int i) {  // of any type
    const at::Tensor* t = tensor(i);
    return t ? t->data_ptr() : nullptr;
  }
  int64_t i64(int i) {
    const long long v = PyLong_AsLongLong(a[i]);
    if (v == -1 && PyErr_Occurred()) {
      PyErr_Clear();
      ok = false;
    }
    return v;
  }
  int32_t i32(int i) {
    const int64_t v = i64(i);
    if (v != static_cast<int32_t>(v)) ok = false;
    return static_cast<int32_t>(v);
  }
  float f32(int i) {
    const double v = PyFloat_AsDouble(a[i]);
    if (v == -1.0 && PyErr_Occurred()) {
      PyErr_Clear();
      ok = false;
    }
    return static_cast<float>(v);
  }
  void* stream(int i) { return reinterpret_cast<void*>(static_cast<uintptr_t>(i64(i))); }
};

// The interpreter's lock let go.
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};
// The status of f(), made without the lock.
template <class F>
PyObject* status(F f) {
  int rc;
  {
    Unlocked unlocked;
    rc = f();
  }
  return PyLong_FromLong(rc);
}
// An entry of N arguments: what F returns, or None where it throws.
template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) Py_RETURN_NONE;
  try {
    return F(args);
  } catch (...) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
}

constexpr auto kBf16 = at::kBFloat16;
constexpr auto kI32 = at::kInt;

// (qkv, q_out or None: in place, num_q_heads, head_dim (read in place only), k_cache, v_cache,
//  positions, slot_mapping, cos_sin, num_kv_heads, block_size, num_blocks, q_weight,
//  k_weight, eps, weight_offset, interleaved, kv_dtype, k_scale, v_scale, stream)
PyObject* norm_rope(PyObject* const* args) {
  Args g{args};
  const at::Tensor* qkv = g.tensor(0);
  if (!qkv || qkv->scalar_type() != kBf16 || qkv->dim() != 2) Py_RETURN_NONE;
  const int64_t T = qkv->size(0), row = qkv->size(1);
  int64_t hq = g.i64(2), d = g.i64(3), out_stride = row;
  void* out = qkv->data_ptr();
  if (args[1] != Py_None) {
    const at::Tensor* q = g.tensor(1);
    if (!q || q->scalar_type() != kBf16 || q->dim() != 3 || q->size(0) != T) Py_RETURN_NONE;
    hq = q->size(1);
    d = q->size(2);
    out = q->data_ptr();
    out_stride = 0;
  }
  void* kc = g.bytes(4);
  void* vc = g.bytes(5);
  const void* pos = g.ptr(6, kI32, T);
  const void* slots = g.ptr(7, kI32, T);
  const at::Tensor* cs = g.tensor(8);
  if (!cs || cs->scalar_type() != at::kFloat || cs->dim() != 2) Py_RETURN_NONE;
  const int64_t hkv = g.i64(9);
  const int32_t bs = g.i32(10), code = g.i32(17);
  const int64_t nb = g.i64(11);
  const void* qw = g.optional(12, kBf16, d);
  const void* kw = g.optional(13, kBf16, d);
  const float eps = g.f32(14), off = g.f32(15), ks = g.f32(18), vs = g.f32(19);
  const int inter = PyObject_IsTrue(args[16]);
  void* st = g.stream(20);
  const int64_t most = INT32_MAX;
  if (!g.ok || inter < 0 || !qw != !kw || hq < 0 || hkv < 0 || d < 0 || hq > most || hkv > most ||
      d > most || T > most || cs->size(0) > most || cs->size(1) > most ||
      row < (hq + 2 * hkv) * d) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
  const void* rows = qkv->data_ptr();
  const float* table = static_cast<const float*>(cs->data_ptr());
  const int32_t top = static_cast<int32_t>(cs->size(0)), rot = static_cast<int32_t>(cs->size(1));
  return status([&] {
    return pd_qk_norm_rope_cache(rows, row, qw, kw, eps, off, table, top, rot, inter,
                                 static_cast<const int32_t*>(pos),
                                 static_cast<const int32_t*>(slots), out, out_stride, kc, vc,
                                 static_cast<int32_t>(T), static_cast<int32_t>(hq),
                                 static_cast<int32_t>(hkv), static_cast<int32_t>(d), bs, nb, code,
                                 ks, vs, st);
  });
}

// (q, out, num_q_heads, head_dim, cu_q, tree_mask or None, k_cache, v_cache, block_tables,
//  seq_lens, max_q_len, num_kv_heads, block_size, num_blocks, scale, sliding_window, num_sinks,
//  kv_dtype, k_scale, v_scale, workspace, stream): q and out [total_q, row] with ROWS, else
//  [total_q, num_q_heads, head_dim] and None for the two numbers
template <bool ROWS>
PyObject* decode_tree(PyObject* const* args) {
  Args g{args};
  const at::Tensor* q = g.tensor(0);
  const at::Tensor* o = g.tensor(1);
  if (!g.ok || q->scalar_type() != kBf16 || o->scalar_type() != kBf16 ||
      q->dim() != (ROWS ? 2 : 3) || o->dim() != q->dim() || o->size(0) != q->size(0))
    Py_RETURN_NONE;
  const int64_t T = q->size(0);
  int64_t hq, d, qs = 0, os = 0;
  if constexpr (ROWS) {
    hq = g.i64(2);
    d = g.i64(3);
    qs = q->size(1);
    os = o->size(1);
    if (!g.ok || hq < 0 || d < 0 || hq > INT32_MAX || d > INT32_MAX || qs < hq * d || os < hq * d)
      Py_RETURN_NONE;
  } else {
    if (args[2] != Py_None || args[3] != Py_None || !q->sizes().equals(o->sizes())) Py_RETURN_NONE;
    hq = q->size(1);
    d = q->size(2);
  }
  const at::Tensor* bt = g.tensor(8);
  if (!bt || bt->scalar_type() != kI32 || bt->dim() != 2) Py_RETURN_NONE;
  const int64_t B = bt->size(0), mbs = bt->size(1);
  const void* cu = g.ptr(4, kI32, B + 1);
  const void* mask = g.optional(5, at::kLong, T);
  const void* kc = g.bytes(6);
  const void* vc = g.bytes(7);
  const void* lens = g.ptr(9, kI32, B);
  const int32_t most_q = g.i32(10), hkv = g.i32(11), bs = g.i32(12);
  const int64_t nb = g.i64(13);
  const float scale = g.f32(14), ks = g.f32(18), vs = g.f32(19);
  const int32_t window = g.i32(15), sinks = g.i32(16), code = g.i32(17);
  const at::Tensor* ws = g.tensor(20);
  void* st = g.stream(21);
  const int64_t most = INT32_MAX;
  if (!g.ok || B > most || mbs > most || T > most || hq > most || d > most) Py_RETURN_NONE;
  const void* qp = q->data_ptr();
  void* op = o->data_ptr();
  const void* tables = bt->data_ptr();
  void* work = ws->data_ptr();
  const size_t work_bytes = ws->nbytes();
  return status([&] {
    return pd_decode_tree(qp, qs, static_cast<const int32_t*>(cu),
                          static_cast<const uint64_t*>(mask), kc, vc,
                          static_cast<const int32_t*>(tables), static_cast<const int32_t*>(lens),
                          op, os, static_cast<int32_t>(B), static_cast<int32_t>(T), most_q,
                          static_cast<int32_t>(hq), hkv, static_cast<int32_t>(d), bs,
                          static_cast<int32_t>(mbs), nb, scale, window, sinks, code, ks, vs, work,
                          work_bytes, st);
  });
}

// (k_caches, v_caches, block_tables, seq_lens, cu_q, accepted, num_accepted, new_seq_lens,
//  num_kv_heads, head_dim, block_size, num_blocks, kv_dtype, stream)
PyObject* compact_tree(PyObject* const* args) {
  Args g{args};
  const at::Tensor* k = g.tensor(0);
  const at::Tensor* v = g.tensor(1);
  const at::Tensor* bt = g.tensor(2);
  const at::Tensor* acc = g.tensor(5);
  if (!g.ok || (k->dim() != 1 && k->dim() != 2) || !k->sizes().equals(v->sizes()) ||
      bt->dim() != 2 || bt->scalar_type() != kI32 || acc->dim() != 2 ||
      acc->scalar_type() != kI32 || acc->size(0) != bt->size(0))
    Py_RETURN_NONE;
  const int64_t B = bt->size(0), mbs = bt->size(1), deep = acc->size(1);
  const int64_t layers = k->dim() == 2 ? k->size(0) : 1;
  const int64_t layer_bytes = k->size(k->dim() - 1) * static_cast<int64_t>(k->element_size());
  const void* lens = g.ptr(3, kI32, B);
  const void* cu = g.ptr(4, kI32, B + 1);
  const void* num = g.ptr(6, kI32, B);
  void* new_lens = g.ptr(7, kI32, B);
  const int32_t hkv = g.i32(8), d = g.i32(9), bs = g.i32(10), code = g.i32(12);
  const int64_t nb = g.i64(11), most = INT32_MAX;
  void* st = g.stream(13);
  if (!g.ok || B > most || mbs > most || deep > most || layers > most) Py_RETURN_NONE;
  void* kp = k->data_ptr();
  void* vp = v->data_ptr();
  const void* tables = bt->data_ptr();
  const void* accepted = acc->data_ptr();
  return status([&] {
    return pd_compact_tree(kp, vp, layer_bytes, static_cast<int32_t>(layers),
                           static_cast<const int32_t*>(tables), static_cast<const int32_t*>(lens),
                           static_cast<const int32_t*>(cu), static_cast<const int32_t*>(accepted),
                           static_cast<const int32_t*>(num), static_cast<int32_t>(deep),
                           static_cast<int32_t*>(new_lens), static_cast<int32_t>(B), hkv, d, bs,
                           static_cast<int32_t>(mbs), nb, code, st);
  });
}

// A method of N arguments.
template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<F, N>)),
          METH_FASTCALL, nullptr};
}
PyMethodDef methods[] = {method<norm_rope, 21>("norm_rope"),
                         method<decode_tree<false>, 22>("decode_tree"),
                         method<decode_tree<true>, 22>("decode_tree_rows"),
                         method<compact_tree, 14>("compact_tree"),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods,
                      nullptr,               nullptr,    nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
