// Host side of libttcff: the C ABI declared in include/gemm_ff.h.  Arguments are
// checked here, in the order and with the codes of mx_api.cu; the kernels are
// launched by the other ff_*.cu files.
#include <cuda_runtime.h>
#include <stdint.h>

#include <initializer_list>

#include "extent.h"
#include "ff_internal.h"

namespace ttc {
namespace ff {
namespace {

// (tiles of 256 rows are counted in 32 bits)
bool size_ok(int64_t n) { return n >= 0 && n <= INT32_MAX - 255; }
bool dtype_ok(int t) { return t == MX_F16 || t == MX_BF16; }
bool act_ok(int a) { return a >= GEMM_ACT_NONE && a <= FF_ACT_SILU; }

int check_bytes(const void* p, uint64_t span, int device) {
  if (p == nullptr) return GEMM_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(p) & 15u) != 0) return GEMM_ERR_ALIGNMENT;
  return check_device_range(p, device, span);
}

// A matrix of elements of `unit` bytes whose rows start on 16 bytes.
int check_matrix(const void* p, int64_t rows, int64_t cols, int64_t ld, int unit, int device) {
  if (p == nullptr || ld < cols || ld >= (1ll << 40) / unit) return GEMM_ERR_INVALID_ARG;
  if ((ld * unit & 15) != 0) return GEMM_ERR_ALIGNMENT;
  return check_bytes(p, matrix_span(rows, cols, ld, unit), device);
}

// No two outputs, and no output and input, are the same matrix.
bool distinct(std::initializer_list<const void*> outputs,
              std::initializer_list<const void*> inputs) {
  for (auto o = outputs.begin(); o != outputs.end(); ++o) {
    if (*o == nullptr) continue;
    for (auto other = outputs.begin(); other != o; ++other)
      if (*other == *o) return false;
    for (const void* i : inputs)
      if (i == *o) return false;
  }
  return true;
}

int fill_zeros(void* p, int64_t rows, int64_t cols, int64_t ld, cudaStream_t stream) {
  const cudaError_t e =
      cudaMemset2DAsync(p, static_cast<size_t>(ld) * 2, 0, static_cast<size_t>(cols) * 2,
                        static_cast<size_t>(rows), stream);
  return e == cudaSuccess ? GEMM_OK : runtime_error();
}

// The pair kernel takes a product of more than 64 rows whose tiles of 256 x `cols` are at least
// a quarter as many as the SMs (each tile takes two), and all weight gradients.  Measured, pair
// and split kernel:
//   gated    128 tiles (1000 x 4096 -> 4096) 48.7 and 92.7 us, 112 (96 x 4096 -> 14336) 51.1 and
//            52.1, 64 (512 x 1024 -> 4096) 10.9 and 23.8; 32 tiles: 24.6 and 25.0 (256 x 4096 ->
//            4096), 9.8 and 11.9 (1000 x 1024 -> 1000), but 24.1 and 16.5 (96 x 4096 -> 4096);
//            16 (512 x 1024 -> 1000) 9.4 and 9.2, 8 (128 x 1024 -> 1000) 9.3 and 7.3
//   dX       64 tiles (1000 x 4096 <- 14336) 193.7 and 267.3, 32 (512 x 4096 <- 4096) 48.2 and
//            45.2, 16 (1000 x 1024 <- 4096) 50.7 and 33.7
//   64 rows  112 tiles (64 x 4096 -> 14336, gated) 50.4 and 40.7
int run_product(const Product& p, const DeviceCtx& d) {
  const int64_t cols = p.form == kGated ? 128 : 256;
  const int64_t pair_tiles = (p.M + 255) / 256 * ((p.N + cols - 1) / cols);
  if (p.form == kStack || (p.M > 64 && pair_tiles >= d.sm_count / 4))
    return launch_pair_product(p, d);
  return launch_split_product(p, d);
}

int run_gated(const Product& p) {
  if (!size_ok(p.M) || !size_ok(p.N) || !size_ok(p.K) || !dtype_ok(p.dtype) || !act_ok(p.act) ||
      (p.gate == nullptr) != (p.up == nullptr))
    return GEMM_ERR_INVALID_ARG;
  if (p.M == 0 || p.N == 0) return GEMM_OK;
  DeviceCtx d;
  int rc = get_device(&d);
  if (rc != GEMM_OK) return rc;
  load_entry_points();
  if (!distinct({p.C[0].p, p.gate, p.up}, {p.A[0].p, p.B[0].p, p.B[1].p}))
    return GEMM_ERR_INVALID_ARG;
  rc = check_matrix(p.C[0].p, p.M, p.N, p.C[0].ld, 2, d.device);
  if (rc == GEMM_OK && p.gate != nullptr) {
    rc = check_matrix(p.gate, p.M, p.N, p.ld_gate, 4, d.device);
    if (rc == GEMM_OK) rc = check_matrix(p.up, p.M, p.N, p.ld_up, 4, d.device);
  }
  if (rc != GEMM_OK) return rc;
  if (p.K == 0) {  // sums over nothing: act(0) * 0 = 0
    rc = fill_zeros(const_cast<void*>(p.C[0].p), p.M, p.N, p.C[0].ld, p.stream);
    if (rc == GEMM_OK && p.gate != nullptr) {
      rc = fill_zeros(p.gate, p.M, 2 * p.N, 2 * p.ld_gate, p.stream);
      if (rc == GEMM_OK) rc = fill_zeros(p.up, p.M, 2 * p.N, 2 * p.ld_up, p.stream);
    }
    return rc;
  }
  rc = check_matrix(p.A[0].p, p.M, p.K, p.A[0].ld, 2, d.device);
  for (int i = 0; i < 2 && rc == GEMM_OK; ++i)
    rc = check_matrix(p.B[i].p, p.N, p.K, p.B[i].ld, 2, d.device);
  return rc == GEMM_OK ? run_product(p, d) : rc;
}

int check_w4(const W4Weight& w, int64_t rows, int64_t cols, int group, int device) {
  const int64_t groups = (cols + group - 1) / group;
  int rc = check_matrix(w.Q, rows, (cols + 7) / 8 * 4, w.ldq, 1, device);
  if (rc == GEMM_OK) rc = check_matrix(w.S, groups, rows, w.lds, 2, device);
  if (rc == GEMM_OK && w.Z != nullptr) rc = check_matrix(w.Z, groups, rows, w.ldz, 1, device);
  return rc;
}

int run_w4(const W4Problem& p) {
  if (!size_ok(p.M) || !size_ok(p.N) || !size_ok(p.K) || !dtype_ok(p.dtype) || !act_ok(p.act) ||
      (p.group != 32 && p.group != 64 && p.group != 128) ||
      (p.gated && (p.w[0].Z == nullptr) != (p.w[1].Z == nullptr)))
    return GEMM_ERR_INVALID_ARG;
  if (p.M == 0 || p.N == 0) return GEMM_OK;
  DeviceCtx d;
  int rc = get_device(&d);
  if (rc != GEMM_OK) return rc;
  load_entry_points();
  if (!distinct({p.Y}, {p.X, p.bias, p.w[0].Q, p.w[0].S, p.w[0].Z, p.w[1].Q, p.w[1].S, p.w[1].Z}))
    return GEMM_ERR_INVALID_ARG;
  rc = check_matrix(p.Y, p.M, p.N, p.ldy, 2, d.device);
  if (rc == GEMM_OK && p.bias != nullptr)
    rc = check_bytes(p.bias, 2u * static_cast<uint64_t>(p.N), d.device);
  if (rc != GEMM_OK) return rc;
  if (p.K == 0)
    return p.gated ? fill_zeros(p.Y, p.M, p.N, p.ldy, p.stream)
                   : launch_bias_fill(p.bias, p.Y, p.M, p.N, p.ldy, p.dtype, p.act, p.stream);
  rc = check_matrix(p.X, p.M, p.K, p.ldx, 2, d.device);
  for (int i = 0; i < (p.gated ? 2 : 1) && rc == GEMM_OK; ++i)
    rc = check_w4(p.w[i], p.N, p.K, p.group, d.device);
  return rc == GEMM_OK ? launch_w4(p, d) : rc;
}

}  // namespace
}  // namespace ff
}  // namespace ttc

using namespace ttc;
using namespace ttc::ff;

extern "C" {

int ff_abi_version(void) { return 10000; }

int ff_gated(const void* X, const void* Wg, const void* Wu, void* H, void* G, void* U, int64_t M,
             int64_t F, int64_t D, int64_t ldx, int64_t ldwg, int64_t ldwu, int64_t ldh,
             int64_t ldg, int64_t ldu, int dtype, int activation, gemm_stream_t stream) {
  Product p{};
  p.form = kGated;
  p.A[0] = p.A[1] = {X, ldx};
  p.B[0] = {Wg, ldwg};
  p.B[1] = {Wu, ldwu};
  p.C[0] = {H, ldh};
  p.gate = static_cast<float*>(G);
  p.up = static_cast<float*>(U);
  p.ld_gate = ldg;
  p.ld_up = ldu;
  p.M = M;
  p.N = F;
  p.K = D;
  p.dtype = dtype;
  p.act = activation;
  p.stream = stream;
  return run_gated(p);
}

int ff_gated_backward(const void* dH, const void* X, const void* Wg, const void* Wu, const void* G,
                      const void* U, void* dG, void* dU, void* dX, void* dWg, void* dWu, int64_t M,
                      int64_t F, int64_t D, int64_t lddh, int64_t ldx, int64_t ldwg, int64_t ldwu,
                      int64_t ldg, int64_t ldu, int64_t lddg, int64_t lddu, int64_t lddx,
                      int64_t lddwg, int64_t lddwu, int dtype, int activation,
                      gemm_stream_t stream) {
  if (!size_ok(M) || !size_ok(F) || !size_ok(D) || !dtype_ok(dtype) || !act_ok(activation) ||
      (dWg == nullptr) != (dWu == nullptr))
    return GEMM_ERR_INVALID_ARG;
  const bool want_x = dX != nullptr && M > 0 && D > 0;
  const bool want_w = dWg != nullptr && F > 0 && D > 0;
  const bool any = M > 0 && F > 0;  // there are sums to take
  if (!any && !want_x && !want_w) return GEMM_OK;
  DeviceCtx d;
  int rc = get_device(&d);
  if (rc != GEMM_OK) return rc;
  load_entry_points();
  if (!distinct({dG, dU, dX, dWg, dWu}, {dH, X, Wg, Wu, G, U})) return GEMM_ERR_INVALID_ARG;
  if (any) {
    rc = check_matrix(dH, M, F, lddh, 2, d.device);
    if (rc == GEMM_OK) rc = check_matrix(G, M, F, ldg, 4, d.device);
    if (rc == GEMM_OK) rc = check_matrix(U, M, F, ldu, 4, d.device);
    if (rc == GEMM_OK) rc = check_matrix(dG, M, F, lddg, 2, d.device);
    if (rc == GEMM_OK) rc = check_matrix(dU, M, F, lddu, 2, d.device);
  }
  if (rc == GEMM_OK && want_x) rc = check_matrix(dX, M, D, lddx, 2, d.device);
  if (rc == GEMM_OK && want_x && any) {
    rc = check_matrix(Wg, F, D, ldwg, 2, d.device);
    if (rc == GEMM_OK) rc = check_matrix(Wu, F, D, ldwu, 2, d.device);
  }
  if (rc == GEMM_OK && want_w) {
    rc = check_matrix(dWg, F, D, lddwg, 2, d.device);
    if (rc == GEMM_OK) rc = check_matrix(dWu, F, D, lddwu, 2, d.device);
    if (rc == GEMM_OK && any) rc = check_matrix(X, M, D, ldx, 2, d.device);
  }
  if (rc != GEMM_OK) return rc;
  if (!any) {  // sums over nothing
    if (want_x) rc = fill_zeros(dX, M, D, lddx, stream);
    if (rc == GEMM_OK && want_w) rc = fill_zeros(dWg, F, D, lddwg, stream);
    if (rc == GEMM_OK && want_w) rc = fill_zeros(dWu, F, D, lddwu, stream);
    return rc;
  }
  rc = launch_slope(SlopeProblem{dH, static_cast<const float*>(G), static_cast<const float*>(U), dG,
                                 dU, M, F, lddh, ldg, ldu, lddg, lddu, dtype, activation, stream},
                    d);
  Product p{};
  p.A[0] = {dG, lddg};
  p.A[1] = {dU, lddu};
  p.dtype = dtype;
  p.stream = stream;
  if (rc == GEMM_OK && want_x) {
    p.form = kConcat;
    p.B[0] = {Wg, ldwg};
    p.B[1] = {Wu, ldwu};
    p.C[0] = p.C[1] = {dX, lddx};
    p.M = M;
    p.N = D;
    p.K = F;
    rc = run_product(p, d);
  }
  if (rc == GEMM_OK && want_w) {
    p.form = kStack;
    p.B[0] = p.B[1] = {X, ldx};
    p.C[0] = {dWg, lddwg};
    p.C[1] = {dWu, lddwu};
    p.M = F;
    p.N = D;
    p.K = M;
    rc = run_product(p, d);
  }
  return rc;
}

int ff_w4_gemm(const void* X, const void* Q, const void* S, const void* Z, const void* bias,
               void* Y, int64_t M, int64_t N, int64_t K, int64_t ldx, int64_t ldq, int64_t lds,
               int64_t ldz, int64_t ldy, int group, int dtype, int activation,
               gemm_stream_t stream) {
  W4Problem p{};
  p.X = X;
  p.bias = bias;
  p.w[0] = {Q, S, Z, ldq, lds, ldz};
  p.Y = Y;
  p.M = M;
  p.N = N;
  p.K = K;
  p.ldx = ldx;
  p.ldy = ldy;
  p.group = group;
  p.dtype = dtype;
  p.act = activation;
  p.stream = stream;
  return run_w4(p);
}

int ff_w4_gated(const void* X, const void* Qg, const void* Sg, const void* Zg, const void* Qu,
                const void* Su, const void* Zu, void* H, int64_t M, int64_t F, int64_t D,
                int64_t ldx, int64_t ldqg, int64_t ldsg, int64_t ldzg, int64_t ldqu, int64_t ldsu,
                int64_t ldzu, int64_t ldh, int group, int dtype, int activation,
                gemm_stream_t stream) {
  W4Problem p{};
  p.X = X;
  p.w[0] = {Qg, Sg, Zg, ldqg, ldsg, ldzg};
  p.w[1] = {Qu, Su, Zu, ldqu, ldsu, ldzu};
  p.Y = H;
  p.M = M;
  p.N = F;
  p.K = D;
  p.ldx = ldx;
  p.ldy = ldh;
  p.group = group;
  p.dtype = dtype;
  p.act = activation;
  p.gated = true;
  p.stream = stream;
  return run_w4(p);
}

int ff_get_device_status(gemm_stream_t stream, int* device_status) {
  if (device_status == nullptr) return GEMM_ERR_INVALID_ARG;
  DeviceCtx d;
  const int rc = get_device(&d);
  if (rc != GEMM_OK) return rc;
  int host = 0;
  if (cudaMemcpyAsync(&host, d.status, sizeof(int), cudaMemcpyDeviceToHost, stream) !=
          cudaSuccess ||
      cudaStreamSynchronize(stream) != cudaSuccess)
    return runtime_error();
  if (host != 0 && (cudaMemsetAsync(d.status, 0, sizeof(int), stream) != cudaSuccess ||
                    cudaStreamSynchronize(stream) != cudaSuccess))
    return runtime_error();
  *device_status = host;
  return GEMM_OK;
}

}  // extern "C"
