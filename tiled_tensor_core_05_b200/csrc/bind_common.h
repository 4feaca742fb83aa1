// What the CPython bindings share: argument checks, the device and stream of a
// call, outputs, and the way of an error from here to Python.
#pragma once

#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <utility>

#include "../../include/gemm_mx.h"

namespace {

struct PyError {};  // a Python exception is set

[[noreturn]] void fail(PyObject* type, const char* format, const char* what, int64_t a = 0,
                       int64_t b = 0) {
  PyErr_Format(type, format, what, static_cast<long long>(a), static_cast<long long>(b));
  throw PyError{};
}

const at::Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) fail(PyExc_TypeError, "%s must be a tensor", what);
  return THPVariable_Unpack(o);
}

int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw PyError{};
  return v;
}

// A code of an activation or a format: what no int holds is none, -1, which the libraries refuse.
int code(PyObject* o) {
  const int64_t v = integer(o);
  return v == static_cast<int>(v) ? static_cast<int>(v) : -1;
}

// Code of the 16-bit type of a CUDA tensor.
int dtype_of(const at::Tensor& t, const char* what) {
  const auto s = t.scalar_type();
  if (s != at::kHalf && s != at::kBFloat16)
    fail(PyExc_TypeError, "%s must be a torch.float16 or torch.bfloat16 tensor", what);
  if (!t.is_cuda()) fail(PyExc_ValueError, "%s must be a CUDA tensor", what);
  return s == at::kHalf ? MX_F16 : MX_BF16;
}

// Checks a matrix; its row stride in elements (of a single row, whose stride
// means nothing, the columns rounded up to 8).
int64_t matrix(const at::Tensor& t, const char* what, int64_t rows, int64_t cols,
               at::ScalarType type, at::Device device) {
  if (t.scalar_type() != type) fail(PyExc_TypeError, "%s has another type than x or out", what);
  if (t.dim() != 2 || t.size(0) != rows || t.size(1) != cols)
    fail(PyExc_ValueError, "%s must be a matrix (%lld, %lld)", what, rows, cols);
  if (t.device() != device) fail(PyExc_ValueError, "%s is on another device", what);
  if (t.stride(1) != 1 && cols > 1)
    fail(PyExc_ValueError, "the columns of %s must be contiguous (stride(1) == 1)", what);
  return rows > 1 ? t.stride(0) : (cols + 7) / 8 * 8;
}

const void* vector(const at::Tensor& t, const char* what, int64_t n, at::ScalarType type,
                   at::Device device) {
  if (t.scalar_type() != type) fail(PyExc_TypeError, "%s has another type than x or out", what);
  if (t.numel() != n || !t.is_contiguous() || t.device() != device)
    fail(PyExc_ValueError, "%s must be %lld contiguous values on the same device", what, n);
  return t.data_ptr();
}

// The device of a call is current inside one of these, and so is the stream
// that writes its outputs: new memory belongs to that stream.
class Context {
 public:
  Context(at::Device device, PyObject* stream) : guard_(device) {
    if (stream == Py_None) {
      handle_ = c10::cuda::getCurrentCUDAStream(device.index()).stream();
    } else {
      handle_ = static_cast<cudaStream_t>(PyLong_AsVoidPtr(stream));
      if (PyErr_Occurred()) throw PyError{};
      stream_.emplace(c10::cuda::getStreamFromExternal(handle_, device.index()));
    }
  }
  gemm_stream_t handle() const { return handle_; }

 private:
  c10::cuda::CUDAGuard guard_;
  std::optional<c10::cuda::CUDAStreamGuard> stream_;
  cudaStream_t handle_;
};

// A new matrix whose rows start on 16 bytes.
at::Tensor new_matrix(int64_t rows, int64_t cols, at::ScalarType type, at::Device device) {
  const auto o = at::TensorOptions(device).dtype(type);
  if (cols % 8 == 0) return at::empty({rows, cols}, o);
  return at::empty_strided({rows, cols}, {(cols + 7) / 8 * 8, 1}, o);
}

PyObject* wrap(const at::Tensor& t) { return THPVariable_Wrap(t); }

void expect(Py_ssize_t got, Py_ssize_t want) {
  if (got != want) fail(PyExc_TypeError, "%s takes %lld arguments", "the call", want);
}

template <class F>
int call(F&& f) {
  int rc;
  Py_BEGIN_ALLOW_THREADS rc = f();
  Py_END_ALLOW_THREADS return rc;
}

template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    return F(args, n);
  } catch (const PyError&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<F>)),
          METH_FASTCALL, nullptr};
}

}  // namespace
