// What the native sides of the Python bindings share: reading arguments and
// tensors, refusing with a Python exception, and calling with the tensors' device
// current.
#pragma once

#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <string>

#include "nvfp4.h"

namespace nvfp4_bind {

// torch's accessors, fetched once
inline PyObject* get_device = nullptr;       // torch._C._cuda_getDevice
inline PyObject* exchange_device = nullptr;  // torch._C._cuda_exchangeDevice
inline PyObject* raw_stream = nullptr;       // torch._C._cuda_getCurrentRawStream

struct Refused {};  // a Python exception is set

[[noreturn]] inline void refuse(const char* format, ...) {
  va_list args;
  va_start(args, format);
  PyErr_FormatV(PyExc_ValueError, format, args);
  va_end(args);
  throw Refused();
}

inline std::string shape_of(const at::Tensor& t) {
  std::string s = "(";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + (t.dim() == 1 ? ",)" : ")");
}

inline const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s must be a tensor, got %s", name, Py_TYPE(o)->tp_name);
    throw Refused();
  }
  return THPVariable_Unpack(o);
}

inline void on_device(const at::Tensor& t, const char* name, const at::Tensor& like) {
  if (t.device() != like.device())
    refuse("%s is on %s, expected %s", name, t.device().str().c_str(), like.device().str().c_str());
}

inline int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused();
  return v;
}

inline int32_t dtype_code(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kFloat: return NVFP4_F32;
    case at::kBFloat16: return NVFP4_BF16;
    case at::kHalf: return NVFP4_F16;
    default:
      PyErr_Format(PyExc_TypeError, "unsupported dtype %s", at::toString(t.scalar_type()));
      throw Refused();
  }
}

// a dense int32 tensor [n]
inline int32_t* ints(PyObject* o, int64_t n, const char* name, const at::Tensor& like) {
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != at::kInt) refuse("%s must be int32, got %s", name, at::toString(t.scalar_type()));
  if (t.dim() != 1 || t.size(0) != n)
    refuse("%s must have shape (%lld,), got %s", name, (long long)n, shape_of(t).c_str());
  if (!t.is_contiguous()) refuse("%s must be contiguous", name);
  on_device(t, name, like);
  return static_cast<int32_t*>(t.data_ptr());
}

// a one-element float32 tensor
inline const float* scale(PyObject* o, const char* name, const at::Tensor& like) {
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != at::kFloat || t.numel() != 1)
    refuse("%s must be a float32 tensor with one element, got %s with %lld", name, at::toString(t.scalar_type()),
           (long long)t.numel());
  on_device(t, name, like);
  return static_cast<const float*>(t.data_ptr());
}

// [tokens][heads][head_dim] with any strides between heads and tokens; the stride of an axis of one is free
struct Heads {
  void* p;
  int64_t tokens, heads, dim, token, head;
  Heads() : p(nullptr), tokens(0), heads(0), dim(0), token(0), head(0) {}
  Heads(PyObject* o, const char* name, const at::Tensor& like, const at::Tensor* same = nullptr) {
    const at::Tensor& t = tensor(o, name);
    if (t.scalar_type() != like.scalar_type() || (same && t.sizes() != same->sizes()))
      refuse("%s must be %s of shape %s, got %s %s", name, at::toString(like.scalar_type()),
             shape_of(same ? *same : like).c_str(), at::toString(t.scalar_type()), shape_of(t).c_str());
    if (t.dim() != 3) refuse("%s must be [tokens, heads, head_dim], got %s", name, shape_of(t).c_str());
    on_device(t, name, like);
    tokens = t.size(0);
    heads = t.size(1);
    dim = t.size(2);
    if (t.stride(2) != 1 && dim != 1) refuse("%s must have unit stride along head_dim", name);
    head = heads > 1 ? t.stride(1) : dim;
    token = tokens > 1 ? t.stride(0) : heads * head;
    p = t.data_ptr();
  }
};

inline int64_t call1(PyObject* f, int64_t v) {
  PyObject* arg = PyLong_FromLongLong(v);
  PyObject* r = arg ? PyObject_CallOneArg(f, arg) : nullptr;
  Py_XDECREF(arg);
  if (!r) throw Refused();
  const int64_t got = PyLong_AsLongLong(r);
  Py_DECREF(r);
  if (got == -1 && PyErr_Occurred()) throw Refused();
  return got;
}

// `call(stream)` with the tensors' device current
template <typename F>
PyObject* launch(const char* name, const at::Tensor& like, PyObject* stream, F call) {
  if (!like.is_cuda()) refuse("%s needs GPU tensors", name);
  const int64_t index = like.get_device();
  PyObject* now = PyObject_CallNoArgs(get_device);
  if (!now) throw Refused();
  const int64_t current = PyLong_AsLongLong(now);
  Py_DECREF(now);
  void* queue = reinterpret_cast<void*>(stream == Py_None ? call1(raw_stream, index) : integer(stream));
  if (current != index) call1(exchange_device, index);
  const int status = call(queue);
  if (current != index) call1(exchange_device, current);
  return PyLong_FromLong(status);
}

inline void count(Py_ssize_t got, Py_ssize_t want) {
  if (got != want) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, got);
    throw Refused();
  }
}

// no C++ exception leaves a function of the module
template <typename F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (const Refused&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}


// the gated delta layer's functions (gdn_bind.cpp) in the module's table (kv_bind.cpp)
PyObject* causal_conv(PyObject*, PyObject* const* o, Py_ssize_t n_args);
PyObject* causal_conv_step(PyObject*, PyObject* const* o, Py_ssize_t n_args);
PyObject* gated_delta_chunked(PyObject*, PyObject* const* o, Py_ssize_t n_args);
PyObject* gated_delta_step(PyObject*, PyObject* const* o, Py_ssize_t n_args);
PyObject* group_norm(PyObject*, PyObject* const* o, Py_ssize_t n_args);

}  // namespace nvfp4_bind
