// CPython binding of the microscaled operators: argument checks, allocation of
// outputs and marshalling into the C ABI of include/gemm_mx.h, for the calls
// whose kernels take no longer than such work takes in Python (a norm of one
// token: 2.9 us on the GPU, 7.5 us here and in mx.py on the host; 18 us with the
// checks, torch.empty and ctypes in Python).
// mx.py is the only caller; it hands over the addresses of the library's entry
// points.  Errors of arguments raise here; status codes of the library are
// returned, for mx.py to raise.
#include "bind_common.h"

namespace {

struct Entry {
  decltype(&mx_quantize) quantize;
  decltype(&mx_dequantize) dequantize;
  decltype(&mx_rms_norm) rms_norm;
  decltype(&mx_gemm) gemm;
} g_entry;

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

// (x, format, out.data, out.scales, out.ld, stream) -> (rc, data, scales, ld)
PyObject* quantize(PyObject* const* a, Py_ssize_t n) {
  expect(n, 6);
  const at::Tensor& x = tensor(a[0], "x");
  const int dtype = dtype_of(x, "x"), format = code(a[1]);
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
  const int format = code(a[5]);
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
  const int dtype = dtype_of(x, "x"), format = code(a[5]);
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
  const int format = code(a[9]), act = code(a[11]);
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

PyMethodDef g_methods[] = {method<bind>("bind"),         method<quantize>("quantize"),
                           method<dequantize>("dequantize"), method<rms_norm>("rms_norm"),
                           method<gemm>("gemm"),         {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_mxbind", nullptr, -1, g_methods,
                        nullptr,               nullptr,    nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__mxbind(void) { return PyModule_Create(&g_module); }
