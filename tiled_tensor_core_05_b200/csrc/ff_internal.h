// Host-side declarations shared by the translation units of libttcff.
#pragma once

#include "../../include/gemm_ff.h"
#include "internal.h"
#include "mx_internal.h"

namespace ttc {
namespace ff {

using mx::Launch;
using mx::launched;
using mx::Residency;

// A row-major matrix of 16-bit elements, row stride in elements.
struct Mat {
  const void* p;
  int64_t ld;
};

// 16-bit products that share a launch (all sizes positive and checked):
//   kGated   C[0] = act(A[0] B[0]^T) * (A[0] B[1]^T); gate and up, the fp32
//            projections, are written where they are not null
//   kConcat  C[0] = A[0] B[0] + A[1] B[1]
//   kStack   C[i] = A[i]^T B[0], i = 0, 1
// A is M x K as stored (K x M for kStack), B is N x K (K x N but for kGated).
enum Form { kGated, kConcat, kStack };

struct Product {
  Form form;
  Mat A[2], B[2], C[2];
  float *gate, *up;
  int64_t ld_gate, ld_up;
  int64_t M, N, K;
  int dtype, act;
  cudaStream_t stream;
};

struct SlopeProblem {  // dG and dU from dH and the fp32 projections
  const void* dH;
  const float *G, *U;
  void *dG, *dU;
  int64_t rows, cols, lddh, ldg, ldu, lddg, lddu;
  int dtype, act;
  cudaStream_t stream;
};

struct W4Weight {
  const void *Q, *S, *Z;
  int64_t ldq, lds, ldz;
};

struct W4Problem {
  const void *X, *bias;
  W4Weight w[2];  // the second one for the gated form
  void* Y;
  int64_t M, N, K, ldx, ldy;
  int group, dtype, act;
  bool gated;
  cudaStream_t stream;
};

// Return 0 or a GEMM_ERR_* code.
int launch_pair_product(const Product& p, const DeviceCtx& d);
int launch_split_product(const Product& p, const DeviceCtx& d);
int launch_slope(const SlopeProblem& p, const DeviceCtx& d);
int launch_w4(const W4Problem& p, const DeviceCtx& d);
// The kernel of launch_w4 for very few rows, and whether it takes a product.
bool w4_few_fits(const W4Problem& p);
int launch_w4_few(const W4Problem& p, const DeviceCtx& d);
// Y = act(bias) (act(0) without one): products over no elements
int launch_bias_fill(const void* bias, void* Y, int64_t rows, int64_t cols, int64_t ldy, int dtype,
                     int act, cudaStream_t stream);

}  // namespace ff
}  // namespace ttc
