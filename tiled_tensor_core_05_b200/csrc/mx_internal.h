// Host-side declarations shared by the translation units of libttcmx.
#pragma once

#include <atomic>

#include "../../include/gemm_mx.h"
#include "internal.h"

namespace ttc {
namespace mx {

struct ConvertProblem {
  const void* X;  // 16-bit matrix (written by the dequantiser)
  const void* Q;  // element bytes
  const void* S;  // scale tiles
  int64_t rows, cols, ldx, ldq;
  int dtype, format;
  cudaStream_t stream;
};

struct NormProblem {
  const void *X, *R, *W;
  void *H, *Y, *S;
  int64_t rows, cols, ldx, ldr, ldh, ldy;
  float eps;
  int dtype, format;
  cudaStream_t stream;
};

struct MxGemmProblem {
  const void *A, *SA, *B, *SB, *bias;
  void* C;
  int64_t M, N, K, lda, ldb, ldc;
  int format, dtype, act;
  cudaStream_t stream;
};

// All sizes positive and checked.  Return 0 or a GEMM_ERR_* code.
int launch_quantize(const ConvertProblem& p);
int launch_dequantize(const ConvertProblem& p);
int launch_rms_norm(const NormProblem& p);
int launch_mx_split_gemm(const MxGemmProblem& p, const DeviceCtx& d);
int launch_mx_pair_gemm(const MxGemmProblem& p, const DeviceCtx& d);
int launch_mx_pair_split_gemm(const MxGemmProblem& p, const DeviceCtx& d);
// C = act(bias), or act(0) without one: a product over no elements.
int launch_mx_bias_fill(const MxGemmProblem& p);

// Launch configuration with the programmatic attribute.
struct Launch {
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg;
  Launch(dim3 grid, dim3 block, size_t smem, cudaStream_t stream) : cfg{} {
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = static_cast<unsigned>(pdl_attribute(&attr[0]));
  }
  void cluster(unsigned n) {
    cudaLaunchAttribute& a = attr[cfg.numAttrs++];
    a.id = cudaLaunchAttributeClusterDimension;
    a.val.clusterDim.x = n;
    a.val.clusterDim.y = 1;
    a.val.clusterDim.z = 1;
  }
};

// The status of a launch, by what the launch itself returned.
inline int launched(cudaError_t e) { return e == cudaSuccess ? GEMM_OK : runtime_error(); }

// How many clusters of c CTAs (c = 2 .. 8) of a kernel the GPU holds at one CTA
// an SM, asked once per device: the GPCs leave SMs over.
struct Residency {
  std::atomic<int> clusters[9] = {};  // 0 = not asked yet
  template <class K>
  int of(int c, K kern, int threads, size_t smem, const DeviceCtx& d) {
    int n = clusters[c].load(std::memory_order_relaxed);
    if (n == 0) {
      Launch l(dim3(static_cast<unsigned>(c * d.sm_count)), dim3(static_cast<unsigned>(threads)),
               smem, nullptr);
      l.cluster(static_cast<unsigned>(c));
      if (cudaOccupancyMaxActiveClusters(&n, kern, &l.cfg) != cudaSuccess || n <= 0) {
        cudaGetLastError();
        n = d.sm_count / (c + 1);
      }
      clusters[c].store(n, std::memory_order_relaxed);
    }
    return n;
  }
};

}  // namespace mx
}  // namespace ttc
