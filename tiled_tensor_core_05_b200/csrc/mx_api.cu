// Host side of libttcmx: the C ABI declared in include/gemm_mx.h.  Arguments
// are checked here, in the order and with the codes of gemm_api.cu; the
// kernels are launched by the other mx_*.cu files.
#include <cuda_runtime.h>
#include <stdint.h>

#include "extent.h"
#include "mx_common.cuh"
#include "mx_internal.h"

namespace ttc {
namespace mx {
namespace {

bool size_ok(int64_t n) { return n >= 0 && n <= INT32_MAX; }
bool format_ok(int f) { return f == MX_FP8 || f == MX_FP4; }
bool dtype_ok(int t) { return t == MX_F16 || t == MX_BF16; }

int check_bytes(const void* p, uint64_t span, int device) {
  if (p == nullptr) return GEMM_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(p) & 15u) != 0) return GEMM_ERR_ALIGNMENT;
  return check_device_range(p, device, span);
}

// A matrix of rows of `used` units `ld` units apart, `unit` bytes each; ld a
// multiple of 16 bytes.
int check_rows(const void* p, int64_t rows, int64_t used, int64_t ld, int unit, int device) {
  if (p == nullptr || ld < used || ld >= (1ll << 40) / unit) return GEMM_ERR_INVALID_ARG;
  if ((ld * unit & 15) != 0) return GEMM_ERR_ALIGNMENT;
  return check_bytes(p, matrix_span(rows, used, ld, unit), device);
}

int check_mx(const void* data, const void* scales, int64_t rows, int64_t cols, int64_t ld,
             int format, int device) {
  const int rc = check_rows(data, rows, mx_row_bytes(cols, format), ld, 1, device);
  if (rc != GEMM_OK) return rc;
  return check_bytes(scales, static_cast<uint64_t>(mx_scale_bytes(rows, cols)), device);
}

int check_convert(const ConvertProblem& p) {
  if (!size_ok(p.rows) || !size_ok(p.cols) || !format_ok(p.format) || !dtype_ok(p.dtype))
    return GEMM_ERR_INVALID_ARG;
  if (p.rows == 0 || p.cols == 0) return GEMM_OK;
  DeviceCtx d;
  int rc = get_device(&d);
  if (rc != GEMM_OK) return rc;
  load_entry_points();
  rc = check_rows(p.X, p.rows, p.cols, p.ldx, 2, d.device);
  if (rc != GEMM_OK) return rc;
  return check_mx(p.Q, p.S, p.rows, p.cols, p.ldq, p.format, d.device);
}

int check_norm(const NormProblem& p) {
  if (!size_ok(p.rows) || !size_ok(p.cols) || !dtype_ok(p.dtype) || !(p.eps >= 0.0f) ||
      (p.format != MX_NONE && !format_ok(p.format)))
    return GEMM_ERR_INVALID_ARG;
  if (p.H != nullptr && p.R == nullptr) return GEMM_ERR_INVALID_ARG;
  if (p.rows == 0 || p.cols == 0) return GEMM_OK;
  DeviceCtx d;
  int rc = get_device(&d);
  if (rc != GEMM_OK) return rc;
  load_entry_points();
  rc = check_rows(p.X, p.rows, p.cols, p.ldx, 2, d.device);
  if (rc == GEMM_OK && p.R != nullptr) rc = check_rows(p.R, p.rows, p.cols, p.ldr, 2, d.device);
  if (rc == GEMM_OK && p.H != nullptr) rc = check_rows(p.H, p.rows, p.cols, p.ldh, 2, d.device);
  if (rc == GEMM_OK) rc = check_bytes(p.W, 2u * static_cast<uint64_t>(p.cols), d.device);
  if (rc != GEMM_OK) return rc;
  // updated in place means the same matrix
  if ((p.H != nullptr && p.H == p.X && p.rows > 1 && p.ldh != p.ldx) ||
      (p.H != nullptr && p.H == p.R && p.rows > 1 && p.ldh != p.ldr))
    return GEMM_ERR_INVALID_ARG;
  if (p.Y == p.R || p.Y == p.H || (p.Y == p.X && (p.R != nullptr || p.format != MX_NONE ||
                                                  (p.rows > 1 && p.ldy != p.ldx))))
    return GEMM_ERR_INVALID_ARG;
  if (p.format == MX_NONE) return check_rows(p.Y, p.rows, p.cols, p.ldy, 2, d.device);
  return check_mx(p.Y, p.S, p.rows, p.cols, p.ldy, p.format, d.device);
}

int run_gemm(const MxGemmProblem& p) {
  if (!size_ok(p.M) || !size_ok(p.N) || !size_ok(p.K) || !format_ok(p.format) ||
      !dtype_ok(p.dtype))
    return GEMM_ERR_INVALID_ARG;
  if (p.act != GEMM_ACT_NONE && p.act != GEMM_ACT_RELU && p.act != GEMM_ACT_GELU)
    return GEMM_ERR_INVALID_ARG;
  if (p.M == 0 || p.N == 0) return GEMM_OK;
  DeviceCtx d;
  int rc = get_device(&d);
  if (rc != GEMM_OK) return rc;
  load_entry_points();
  rc = check_rows(p.C, p.M, p.N, p.ldc, 2, d.device);
  if (rc == GEMM_OK && p.bias != nullptr)
    rc = check_bytes(p.bias, 2u * static_cast<uint64_t>(p.N), d.device);
  if (rc != GEMM_OK) return rc;
  if (p.K == 0) return launch_mx_bias_fill(p);
  rc = check_mx(p.A, p.SA, p.M, p.K, p.lda, p.format, d.device);
  if (rc == GEMM_OK) rc = check_mx(p.B, p.SB, p.N, p.K, p.ldb, p.format, d.device);
  if (rc != GEMM_OK) return rc;
  // Measured (us: split kernel, pair kernel, pair tiles with K divided):
  //   1500 x 2000 x 2000 MXFP4 (48 tiles of 256 x 256)   15.9   8.2  14.0
  //   1024 x 4096 x 8192 MXFP8 (64)                      46.8  27.2  38.9
  //   256 x 9000 x 4096 MXFP8 (36)                       16.0  16.8  13.8
  //   256 x 4096 x 8192 MXFP8 (16)                       19.7  24.2  14.3
  //   512 x 2048 x 2048 MXFP4 (16; 8 k-blocks)            6.1   7.3   6.8
  //   128 x 18944 x 4096 MXFP4 (74, half empty)          13.1  13.7  12.8
  //   100 x 28672 x 8192 MXFP4 (112; two waves split)    32.6  28.9  29.6
  // So: the pair kernel where its tiles fill half the SMs, if they are not half
  // empty (M > 128) or the split kernel's would take two waves;
  // else K divided among pairs from 65 rows and 16 k-blocks on; else the split
  // kernel.
  const int64_t pair_tiles = ((p.M + 255) / 256) * ((p.N + 255) / 256);
  const int64_t split_tiles = ((p.M + 63) / 64) * ((p.N + 127) / 128);
  const int64_t num_kb = (mx_row_bytes(p.K, p.format) + 127) / 128;
  if (p.M > 64 && pair_tiles >= d.sm_count / 4 &&
      (p.M > 128 || split_tiles > 2 * d.sm_count))
    return launch_mx_pair_gemm(p, d);
  if (p.M > 64 && num_kb >= 16) return launch_mx_pair_split_gemm(p, d);
  return launch_mx_split_gemm(p, d);
}

}  // namespace
}  // namespace mx
}  // namespace ttc

using namespace ttc;
using namespace ttc::mx;

extern "C" {

int mx_abi_version(void) { return 10000; }

int64_t mx_row_bytes(int64_t cols, int format) {
  if (cols < 0 || !format_ok(format)) return -1;
  return format == MX_FP8 ? cols : cols / 2 + (cols & 1);
}

int64_t mx_scale_bytes(int64_t rows, int64_t cols) {
  if (!size_ok(rows) || !size_ok(cols)) return -1;
  return (rows + kTileRows - 1) / kTileRows * scale_tiles(cols) * kTileBytes;
}

int mx_quantize(const void* X, void* Q, void* S, int64_t rows, int64_t cols, int64_t ldx,
                int64_t ldq, int dtype, int format, gemm_stream_t stream) {
  const ConvertProblem p{X, Q, S, rows, cols, ldx, ldq, dtype, format, stream};
  const int rc = check_convert(p);
  if (rc != GEMM_OK || rows == 0 || cols == 0) return rc;
  return launch_quantize(p);
}

int mx_dequantize(const void* Q, const void* S, void* X, int64_t rows, int64_t cols, int64_t ldq,
                  int64_t ldx, int dtype, int format, gemm_stream_t stream) {
  const ConvertProblem p{X, Q, S, rows, cols, ldx, ldq, dtype, format, stream};
  const int rc = check_convert(p);
  if (rc != GEMM_OK || rows == 0 || cols == 0) return rc;
  return launch_dequantize(p);
}

int mx_rms_norm(const void* X, const void* R, const void* W, void* H, void* Y, void* S,
                int64_t rows, int64_t cols, int64_t ldx, int64_t ldr, int64_t ldh, int64_t ldy,
                float eps, int dtype, int format, gemm_stream_t stream) {
  const NormProblem p{X, R, W, H, Y, S, rows, cols, ldx, ldr, ldh, ldy, eps, dtype, format, stream};
  const int rc = check_norm(p);
  if (rc != GEMM_OK || rows == 0 || cols == 0) return rc;
  return launch_rms_norm(p);
}

int mx_gemm(const void* A, const void* SA, const void* B, const void* SB, const void* bias,
            void* C, int64_t M, int64_t N, int64_t K, int64_t lda, int64_t ldb, int64_t ldc,
            int format, int dtype, int activation, gemm_stream_t stream) {
  return run_gemm(MxGemmProblem{A, SA, B, SB, bias, C, M, N, K, lda, ldb, ldc, format, dtype,
                                activation, stream});
}

int mx_get_device_status(gemm_stream_t stream, int* device_status) {
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
