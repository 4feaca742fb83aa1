// CPython binding of the feed-forward operators (include/gemm_ff.h), in the manner
// of mx_bind.cpp: checks, allocation of outputs and marshalling.  ff.py is the only
// caller; it hands over the addresses of the library's entry points.
#include "../../include/gemm_ff.h"
#include "bind_common.h"

#include <torch/csrc/autograd/functions/basic_ops.h>
#include <torch/csrc/autograd/functions/utils.h>

namespace {

struct Entry {
  decltype(&ff_gated) gated;
  decltype(&ff_gated_backward) gated_backward;
  decltype(&ff_w4_gemm) w4_gemm;
  decltype(&ff_w4_gated) w4_gated;
} g_entry;

// A matrix argument: its address and row stride.
struct Mat {
  void* p = nullptr;
  int64_t ld = 0;
  Mat() = default;
  Mat(const at::Tensor& t, const char* what, int64_t rows, int64_t cols, at::ScalarType type,
      at::Device device)
      : p(t.data_ptr()), ld(matrix(t, what, rows, cols, type, device)) {}
};

PyObject* none() {
  Py_INCREF(Py_None);
  return Py_None;
}

PyObject* wrap_or_none(const at::Tensor& t) { return t.defined() ? wrap(t) : none(); }

struct Input {  // a matrix of activations and what follows from it
  const at::Tensor& t;
  int dtype;
  at::ScalarType type;
  at::Device device;
  int64_t rows, cols;
  Mat m;
  Input(PyObject* o, const char* what)
      : t(tensor(o, what)), dtype(dtype_of(t, what)), type(t.scalar_type()), device(t.device()) {
    if (t.dim() != 2) fail(PyExc_ValueError, "%s must be a matrix", what);
    rows = t.size(0);
    cols = t.size(1);
    m = Mat(t, what, rows, cols, type, device);
  }
};

// These operators record no graph.  Where an input requires a gradient, a backward pass that
// reaches their result raises `message`: without it the gradient would be lost in silence.
// (The node has no edges to the inputs: a result that is kept would keep their gradients'
// accumulators, and with them the stream of this call, for a backward pass captured later.)
// As with torch's own out= forms, a given result (`out`) is refused then, before anything runs.
struct NoGraph {
  std::shared_ptr<torch::autograd::Node> node;
  template <class... Inputs>
  NoGraph(PyObject* out, const char* message, const Inputs&... inputs) {
    if (!torch::autograd::compute_requires_grad(inputs...)) return;
    if (out != Py_None)
      fail(PyExc_RuntimeError, "out= is for inputs that require no gradient: %s", message);
    node = std::make_shared<torch::autograd::Error>(message);
  }
  void mark(const at::Tensor& result) const {
    if (node) torch::autograd::set_history(result, node);
  }
};

int64_t rows_of(const at::Tensor& t, const char* what) {
  if (t.dim() != 2) fail(PyExc_ValueError, "%s must be a matrix", what);
  return t.size(0);
}

// (x, w_gate, w_up, act, out or None, save, stream) -> (rc, h, gate or None, up or None)
PyObject* gated(PyObject* const* a, Py_ssize_t n) {
  expect(n, 7);
  const Input x(a[0], "x");
  const at::Tensor &wg = tensor(a[1], "w_gate"), &wu = tensor(a[2], "w_up");
  const int64_t F = rows_of(wg, "w_gate");
  const Mat mg(wg, "w_gate", F, x.cols, x.type, x.device);
  const Mat mu(wu, "w_up", F, x.cols, x.type, x.device);
  const int act = code(a[3]);
  const bool save = a[5] == Py_True;
  // (with save the caller takes the gradients)
  const NoGraph no_graph(save ? Py_None : a[4],
                         "gemm_gated records no graph: call it with save=True and take the "
                         "gradients from gemm_gated_backward",
                         x.t, wg, wu);
  Context c(x.device, a[6]);
  const at::Tensor h =
      a[4] != Py_None ? tensor(a[4], "out") : new_matrix(x.rows, F, x.type, x.device);
  const Mat mh(h, "out", x.rows, F, x.type, x.device);
  at::Tensor gate, up;
  Mat sg, su;
  if (save) {
    gate = new_matrix(x.rows, F, at::kFloat, x.device);
    up = new_matrix(x.rows, F, at::kFloat, x.device);
    sg = Mat(gate, "gate", x.rows, F, at::kFloat, x.device);
    su = Mat(up, "up", x.rows, F, at::kFloat, x.device);
  }
  const int rc = call([&] {
    return g_entry.gated(x.m.p, mg.p, mu.p, mh.p, sg.p, su.p, x.rows, F, x.cols, x.m.ld, mg.ld,
                         mu.ld, mh.ld, sg.ld, su.ld, x.dtype, act, c.handle());
  });
  if (!save) no_graph.mark(h);
  return Py_BuildValue("iNNN", rc, wrap(h), wrap_or_none(gate), wrap_or_none(up));
}

// (dh, x, w_gate, w_up, gate, up, act, need_x, need_w, stream) -> (rc, dx, dw_gate, dw_up), None
// for what is not needed
PyObject* gated_backward(PyObject* const* a, Py_ssize_t n) {
  expect(n, 10);
  const Input x(a[1], "x");
  const at::Tensor &wg = tensor(a[2], "w_gate"), &wu = tensor(a[3], "w_up");
  const int64_t M = x.rows, D = x.cols, F = rows_of(wg, "w_gate");
  const Mat mg(wg, "w_gate", F, D, x.type, x.device), mu(wu, "w_up", F, D, x.type, x.device);
  const Mat dh(tensor(a[0], "dh"), "dh", M, F, x.type, x.device);
  const Mat g(tensor(a[4], "gate"), "gate", M, F, at::kFloat, x.device);
  const Mat u(tensor(a[5], "up"), "up", M, F, at::kFloat, x.device);
  const int act = code(a[6]);
  Context c(x.device, a[9]);
  const at::Tensor dg = new_matrix(M, F, x.type, x.device), du = new_matrix(M, F, x.type, x.device);
  const Mat mdg(dg, "dg", M, F, x.type, x.device), mdu(du, "du", M, F, x.type, x.device);
  at::Tensor dx, dwg, dwu;
  Mat mdx, mdwg, mdwu;
  if (a[7] == Py_True) {
    dx = new_matrix(M, D, x.type, x.device);
    mdx = Mat(dx, "dx", M, D, x.type, x.device);
  }
  if (a[8] == Py_True) {
    dwg = new_matrix(F, D, x.type, x.device);
    dwu = new_matrix(F, D, x.type, x.device);
    mdwg = Mat(dwg, "dw_gate", F, D, x.type, x.device);
    mdwu = Mat(dwu, "dw_up", F, D, x.type, x.device);
  }
  const int rc = call([&] {
    return g_entry.gated_backward(dh.p, x.m.p, mg.p, mu.p, g.p, u.p, mdg.p, mdu.p, mdx.p, mdwg.p,
                                  mdwu.p, M, F, D, dh.ld, x.m.ld, mg.ld, mu.ld, g.ld, u.ld, mdg.ld,
                                  mdu.ld, mdx.ld, mdwg.ld, mdwu.ld, x.dtype, act, c.handle());
  });
  return Py_BuildValue("iNNN", rc, wrap_or_none(dx), wrap_or_none(dwg), wrap_or_none(dwu));
}

// A 4-bit weight, whose shapes ff.py has checked: data, scales, zeros or None, ld, lds, ldz
struct Weight {
  const void *q, *s, *z = nullptr;
  int64_t ldq, lds, ldz = 0;
  const at::Tensor& scales;
  Weight(PyObject* const* a, const Input& x) : scales(tensor(a[1], "w.scales")) {
    const at::Tensor& data = tensor(a[0], "w.data");
    if (data.device() != x.device) fail(PyExc_ValueError, "%s is on another device", "w");
    if (scales.scalar_type() != x.type)
      fail(PyExc_TypeError, "%s have another type than x", "the scales of w");
    q = data.data_ptr();
    s = scales.data_ptr();
    if (a[2] != Py_None) z = tensor(a[2], "w.zeros").data_ptr();
    ldq = integer(a[3]);
    lds = integer(a[4]);
    ldz = integer(a[5]);
  }
};

// (x, weight: 6, rows, group, bias or None, act, out or None, stream) -> (rc, y)
PyObject* w4_gemm(PyObject* const* a, Py_ssize_t n) {
  expect(n, 13);
  const Input x(a[0], "x");
  const Weight w(a + 1, x);
  const int64_t N = integer(a[7]);
  const int group = code(a[8]), act = code(a[10]);
  const at::Tensor bias_t = a[9] == Py_None ? at::Tensor() : tensor(a[9], "bias");
  const void* bias =
      bias_t.defined() ? vector(bias_t, "bias", N, x.type, x.device) : nullptr;
  const NoGraph no_graph(a[11], "gemm_w4 has no backward pass", x.t, bias_t, w.scales);
  Context c(x.device, a[12]);
  const at::Tensor y =
      a[11] != Py_None ? tensor(a[11], "out") : new_matrix(x.rows, N, x.type, x.device);
  const Mat my(y, "out", x.rows, N, x.type, x.device);
  const int rc = call([&] {
    return g_entry.w4_gemm(x.m.p, w.q, w.s, w.z, bias, my.p, x.rows, N, x.cols, x.m.ld, w.ldq,
                           w.lds, w.ldz, my.ld, group, x.dtype, act, c.handle());
  });
  no_graph.mark(y);
  return Py_BuildValue("iN", rc, wrap(y));
}

// (x, gate weight: 6, up weight: 6, rows, group, act, out or None, stream) -> (rc, h)
PyObject* w4_gated(PyObject* const* a, Py_ssize_t n) {
  expect(n, 18);
  const Input x(a[0], "x");
  const Weight g(a + 1, x), u(a + 7, x);
  const int64_t F = integer(a[13]);
  const int group = code(a[14]), act = code(a[15]);
  const NoGraph no_graph(a[16], "gemm_gated_w4 has no backward pass", x.t, g.scales,
                         u.scales);
  Context c(x.device, a[17]);
  const at::Tensor h =
      a[16] != Py_None ? tensor(a[16], "out") : new_matrix(x.rows, F, x.type, x.device);
  const Mat mh(h, "out", x.rows, F, x.type, x.device);
  const int rc = call([&] {
    return g_entry.w4_gated(x.m.p, g.q, g.s, g.z, u.q, u.s, u.z, mh.p, x.rows, F, x.cols, x.m.ld,
                            g.ldq, g.lds, g.ldz, u.ldq, u.lds, u.ldz, mh.ld, group, x.dtype, act,
                            c.handle());
  });
  no_graph.mark(h);
  return Py_BuildValue("iN", rc, wrap(h));
}

// (addresses of ff_gated, ff_gated_backward, ff_w4_gemm, ff_w4_gated)
PyObject* bind(PyObject* const* a, Py_ssize_t n) {
  expect(n, 4);
  g_entry.gated = reinterpret_cast<decltype(&ff_gated)>(integer(a[0]));
  g_entry.gated_backward = reinterpret_cast<decltype(&ff_gated_backward)>(integer(a[1]));
  g_entry.w4_gemm = reinterpret_cast<decltype(&ff_w4_gemm)>(integer(a[2]));
  g_entry.w4_gated = reinterpret_cast<decltype(&ff_w4_gated)>(integer(a[3]));
  Py_RETURN_NONE;
}

PyMethodDef g_methods[] = {method<bind>("bind"),
                           method<gated>("gated"),
                           method<gated_backward>("gated_backward"),
                           method<w4_gemm>("w4_gemm"),
                           method<w4_gated>("w4_gated"),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_ffbind", nullptr, -1, g_methods,
                        nullptr,               nullptr,    nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ffbind(void) { return PyModule_Create(&g_module); }
