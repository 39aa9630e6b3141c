// What the library's CPython bindings share: tensors checked, results allocated,
// errors raised, streams.
#pragma once
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>
#include <c10/core/TensorImpl.h>
#include <c10/cuda/CUDAStream.h>

#include <cmath>
#include <exception>
#include <string>

#include "qmv.h"

namespace {

PyObject* qmv_error = nullptr;  // the binding's exception class (code, call)

// A Python error is set.
struct Raised {};

[[noreturn]] void value_error(const std::string& s) {
  PyErr_SetString(PyExc_ValueError, s.c_str());
  throw Raised{};
}

void check(int rc, const char* what) {
  if (rc == 0) return;
  PyObject* e = PyObject_CallFunction(qmv_error, "is", rc, what);
  if (e) {
    PyErr_SetObject(qmv_error, e);
    Py_DECREF(e);
  }
  throw Raised{};
}

const at::Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s: a tensor wanted", what);
    throw Raised{};
  }
  return THPVariable_Unpack(o);
}

int dtype_code(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return QMV_DT_F32;
    case at::kHalf: return QMV_DT_F16;
    case at::kBFloat16: return QMV_DT_BF16;
    default: value_error(std::string("float32, float16 or bfloat16 tensor wanted, got ") + c10::toString(t));
  }
}

std::string text(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); i++) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + ")";
}

void on_device(const at::Tensor& t) {
  if (!t.is_cuda()) value_error("tensor must be on a CUDA device");
}

// The address of a contiguous CUDA tensor.
void* ptr(const at::Tensor& t) {
  on_device(t);
  if (!t.is_contiguous()) value_error("tensor must be contiguous");
  return t.data_ptr();
}

// The address of a contiguous CUDA tensor of this type and shape.
void* typed(const at::Tensor& t, at::ScalarType type, at::IntArrayRef shape, const char* what) {
  if (t.scalar_type() != type || t.sizes() != shape)
    value_error(std::string(what) + ": " + c10::toString(type) + " " + text(shape) + " wanted, got " +
                c10::toString(t.scalar_type()) + " " + text(t.sizes()));
  return ptr(t);
}

// The stream of a call: the given one's handle, or torch's current one.
cudaStream_t stream_of(PyObject* o) {
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream().stream();
  const unsigned long long v = PyLong_AsUnsignedLongLong(o);
  if (PyErr_Occurred()) throw Raised{};
  return reinterpret_cast<cudaStream_t>(v);
}

// A new tensor for work on st.  The allocator takes memory for used on the
// current stream: it is told where that is another one, so that memory dropped
// early (a workspace always is) goes to nobody before the work is done.
at::Tensor fresh(at::IntArrayRef shape, at::ScalarType type, const at::Tensor& like, cudaStream_t st) {
  at::Tensor t = at::empty(shape, like.options().dtype(type));
  const c10::DeviceIndex dev = t.device().index();
  if (st != c10::cuda::getCurrentCUDAStream(dev).stream()) t.record_stream(c10::cuda::getStreamFromExternal(st, dev).unwrap());
  return t;
}

// A tensor of its own type over part of buf's memory (which it keeps): results
// that belong together share one allocation, which costs the host more than
// all else of a small call.
at::Tensor piece(const at::Tensor& buf, int64_t byte, at::IntArrayRef shape, at::ScalarType type) {
  auto impl = c10::make_intrusive<c10::TensorImpl>(c10::Storage(buf.storage()), buf.key_set(),
                                                   c10::scalarTypeToTypeMeta(type));
  impl->set_storage_offset(byte / (int64_t)c10::elementSize(type));
  impl->set_sizes_contiguous(shape);
  return at::Tensor(std::move(impl));
}

// A given result, checked, or a new one on like's device.
at::Tensor result(PyObject* o, at::ScalarType type, at::IntArrayRef shape, const at::Tensor& like, cudaStream_t st, const char* what) {
  if (o == Py_None) {
    on_device(like);
    return fresh(shape, type, like, st);
  }
  const at::Tensor& t = tensor(o, what);
  typed(t, type, shape, what);
  return t;
}

long long integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  return v;
}
int as_int(PyObject* o) {
  const long long v = integer(o);
  if (v < INT32_MIN || v > INT32_MAX) value_error("integer out of range");
  return (int)v;
}
double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return v;
}

const int32_t* ints(const at::Tensor& t) {
  if (t.scalar_type() != at::kInt) value_error(std::string("int32 tensor wanted, got ") + c10::toString(t.scalar_type()));
  return static_cast<const int32_t*>(ptr(t));
}

template <class F>
PyObject* guarded(Py_ssize_t got, Py_ssize_t want, F f) {
  if (got != want) {
    PyErr_Format(PyExc_TypeError, "%zd arguments wanted, got %zd", want, got);
    return nullptr;
  }
  try {
    return f();
  } catch (const Raised&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

template <class F>
int called(F f) {
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = f();
  Py_END_ALLOW_THREADS
  return rc;
}

PyObject* wrap(const at::Tensor& t) { return t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None); }

at::Tensor workspace(PyObject* o, size_t bytes, const at::Tensor& like, cudaStream_t st) {
  if (o == Py_None) return fresh({(int64_t)(bytes < 16 ? 16 : bytes)}, at::kByte, like, st);
  const at::Tensor& t = tensor(o, "ws");
  ptr(t);
  return t;
}

#define QMV_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}

}  // namespace
