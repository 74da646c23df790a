// What the modules that marshal torch tensors to libpd.so's calls share: the
// unpacking of arguments, and an entry that declines instead of throwing.
#pragma once

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
// A method of N arguments.
template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<F, N>)),
          METH_FASTCALL, nullptr};
}

constexpr auto kBf16 = at::kBFloat16;
constexpr auto kI32 = at::kInt;
constexpr int64_t kMost = INT32_MAX;

}  // namespace
