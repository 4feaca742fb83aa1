// CPython binding of the microscaled operators: argument checks, allocation of
// outputs and marshalling into the C ABI of include/gemm_mx.h, for the calls
// whose kernels take no longer than such work takes in Python (a norm of one
// token: 2.9 us on the GPU, 7.5 us here and in mx.py on the host; 18 us with the
// checks, torch.empty and ctypes in Python).
// mx.py is the only caller; it hands over the addresses of the library's entry
// points.  Errors of arguments raise here; status codes of the library are
// returned, for mx.py to raise.
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

struct Entry {
  decltype(&mx_quantize) quantize;
  decltype(&mx_dequantize) dequantize;
  decltype(&mx_rms_norm) rms_norm;
  decltype(&mx_gemm) gemm;
} g_entry;

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

int64_t row_bytes(int64_t cols, int format) { return format == MX_FP8 ? cols : (cols + 1) / 2; }

// An MX output: given (checked by the caller) or new.
struct MxOut {
  at::Tensor data, scales;
  int64_t ld;
  MxOut(PyObject* d, PyObject* s, PyObject* given_ld, int64_t rows, int64_t cols, int format,
        at::Device device) {
    if (d != Py_None) {
      data = tensor(d, "out.data");
      scales = tensor(s, "out.scales");
      ld = integer(given_ld);
      return;
    }
    const auto o = at::TensorOptions(device).dtype(at::kByte);
    ld = (row_bytes(cols, format) + 15) / 16 * 16;
    data = at::empty({rows, ld}, o);
    scales = at::empty({(rows + 127) / 128 * ((cols + 127) / 128) * 512}, o);
  }
};

PyObject* wrap(const at::Tensor& t) { return THPVariable_Wrap(t); }

void expect(Py_ssize_t got, Py_ssize_t want) {
  if (got != want) fail(PyExc_TypeError, "%s: wrong number of arguments", "mx");
}

template <class F>
int call(F&& f) {
  int rc;
  Py_BEGIN_ALLOW_THREADS rc = f();
  Py_END_ALLOW_THREADS return rc;
}

// (x, format, out.data, out.scales, out.ld, stream) -> (rc, data, scales, ld)
PyObject* quantize(PyObject* const* a, Py_ssize_t n) {
  expect(n, 6);
  const at::Tensor& x = tensor(a[0], "x");
  const int dtype = dtype_of(x, "x"), format = static_cast<int>(integer(a[1]));
  if (x.dim() != 2) fail(PyExc_ValueError, "%s must be a matrix", "x");
  const int64_t rows = x.size(0), cols = x.size(1);
  const int64_t ldx = matrix(x, "x", rows, cols, x.scalar_type(), x.device());
  Context c(x.device(), a[5]);
  MxOut out(a[2], a[3], a[4], rows, cols, format, x.device());
  const int rc = call([&] {
    return g_entry.quantize(x.data_ptr(), out.data.data_ptr(), out.scales.data_ptr(), rows, cols,
                            ldx, out.ld, dtype, format, c.handle());
  });
  return Py_BuildValue("iNNL", rc, wrap(out.data), wrap(out.scales),
                       static_cast<long long>(out.ld));
}

// (data, scales, rows, cols, ld, format, out or None, type of a new out, stream) -> (rc, out)
PyObject* dequantize(PyObject* const* a, Py_ssize_t n) {
  expect(n, 9);
  const at::Tensor &data = tensor(a[0], "q.data"), &scales = tensor(a[1], "q.scales");
  const int64_t rows = integer(a[2]), cols = integer(a[3]), ld = integer(a[4]);
  const int format = static_cast<int>(integer(a[5]));
  Context c(data.device(), a[8]);
  const at::Tensor out =
      a[6] != Py_None ? tensor(a[6], "out")
                      : new_matrix(rows, cols, integer(a[7]) == MX_F16 ? at::kHalf : at::kBFloat16,
                                   data.device());
  const int dtype = dtype_of(out, "out");
  const int64_t ldx = matrix(out, "out", rows, cols, out.scalar_type(), data.device());
  const int rc = call([&] {
    return g_entry.dequantize(data.data_ptr(), scales.data_ptr(), out.data_ptr(), rows, cols, ld,
                              ldx, dtype, format, c.handle());
  });
  return Py_BuildValue("iN", rc, wrap(out));
}

// (x, weight, eps, residual, residual_out, format, out or out.data, out.scales, out.ld, stream)
// -> (rc, y or data, scales or None, ld, h or None)
PyObject* rms_norm(PyObject* const* a, Py_ssize_t n) {
  expect(n, 10);
  const at::Tensor& x = tensor(a[0], "x");
  const int dtype = dtype_of(x, "x"), format = static_cast<int>(integer(a[5]));
  const auto type = x.scalar_type();
  const at::Device device = x.device();
  if (x.dim() != 2) fail(PyExc_ValueError, "%s must be a matrix", "x");
  const int64_t rows = x.size(0), cols = x.size(1);
  const int64_t ldx = matrix(x, "x", rows, cols, type, device);
  const void* w = vector(tensor(a[1], "weight"), "weight", cols, type, device);
  const double eps = PyFloat_AsDouble(a[2]);
  if (eps == -1.0 && PyErr_Occurred()) throw PyError{};
  Context c(device, a[9]);
  const void* r = nullptr;
  at::Tensor h;
  int64_t ldr = 0, ldh = 0;
  if (a[3] != Py_None) {
    const at::Tensor& t = tensor(a[3], "residual");
    ldr = matrix(t, "residual", rows, cols, type, device);
    r = t.data_ptr();
    h = a[4] != Py_None ? tensor(a[4], "residual_out") : new_matrix(rows, cols, type, device);
    ldh = matrix(h, "residual_out", rows, cols, type, device);
  } else if (a[4] != Py_None) {
    fail(PyExc_ValueError, "%s needs a residual", "residual_out");
  }
  at::Tensor y, s;
  int64_t ldy;
  if (format == MX_NONE) {
    y = a[6] != Py_None ? tensor(a[6], "out") : new_matrix(rows, cols, type, device);
    ldy = matrix(y, "out", rows, cols, type, device);
  } else {
    MxOut out(a[6], a[7], a[8], rows, cols, format, device);
    y = std::move(out.data);
    s = std::move(out.scales);
    ldy = out.ld;
  }
  const int rc = call([&] {
    return g_entry.rms_norm(x.data_ptr(), r, w, h.defined() ? h.data_ptr() : nullptr, y.data_ptr(),
                            s.defined() ? s.data_ptr() : nullptr, rows, cols, ldx, ldr, ldh, ldy,
                            static_cast<float>(eps), dtype, format, c.handle());
  });
  PyObject* none = Py_None;
  Py_INCREF(none);
  Py_INCREF(none);
  PyObject* ps = s.defined() ? (Py_DECREF(none), wrap(s)) : none;
  PyObject* ph = h.defined() ? (Py_DECREF(none), wrap(h)) : none;
  return Py_BuildValue("iNNLN", rc, wrap(y), ps, static_cast<long long>(ldy), ph);
}

// (a.data, a.scales, b.data, b.scales, M, N, K, lda, ldb, format, bias, act, out or None, type of
// a new out, stream) -> (rc, out)
PyObject* gemm(PyObject* const* a, Py_ssize_t n) {
  expect(n, 15);
  const at::Tensor &ad = tensor(a[0], "a.data"), &as = tensor(a[1], "a.scales");
  const at::Tensor &bd = tensor(a[2], "b.data"), &bs = tensor(a[3], "b.scales");
  const int64_t M = integer(a[4]), N = integer(a[5]), K = integer(a[6]);
  const int64_t lda = integer(a[7]), ldb = integer(a[8]);
  const int format = static_cast<int>(integer(a[9])), act = static_cast<int>(integer(a[11]));
  const at::Device device = ad.device();
  Context c(device, a[14]);
  const at::Tensor out =
      a[12] != Py_None ? tensor(a[12], "out")
                       : new_matrix(M, N, integer(a[13]) == MX_F16 ? at::kHalf : at::kBFloat16,
                                    device);
  const int dtype = dtype_of(out, "out");
  const int64_t ldc = matrix(out, "out", M, N, out.scalar_type(), device);
  const void* bias = a[10] == Py_None ? nullptr
                                      : vector(tensor(a[10], "bias"), "bias", N,
                                               out.scalar_type(), device);
  const int rc = call([&] {
    return g_entry.gemm(ad.data_ptr(), as.data_ptr(), bd.data_ptr(), bs.data_ptr(), bias,
                        out.data_ptr(), M, N, K, lda, ldb, ldc, format, dtype, act, c.handle());
  });
  return Py_BuildValue("iN", rc, wrap(out));
}

// (addresses of mx_quantize, mx_dequantize, mx_rms_norm, mx_gemm)
PyObject* bind(PyObject* const* a, Py_ssize_t n) {
  expect(n, 4);
  g_entry.quantize = reinterpret_cast<decltype(&mx_quantize)>(integer(a[0]));
  g_entry.dequantize = reinterpret_cast<decltype(&mx_dequantize)>(integer(a[1]));
  g_entry.rms_norm = reinterpret_cast<decltype(&mx_rms_norm)>(integer(a[2]));
  g_entry.gemm = reinterpret_cast<decltype(&mx_gemm)>(integer(a[3]));
  Py_RETURN_NONE;
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

PyMethodDef g_methods[] = {method<bind>("bind"),         method<quantize>("quantize"),
                           method<dequantize>("dequantize"), method<rms_norm>("rms_norm"),
                           method<gemm>("gemm"),         {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_mxbind", nullptr, -1, g_methods,
                        nullptr,               nullptr,    nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__mxbind(void) { return PyModule_Create(&g_module); }
