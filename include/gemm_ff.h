/*
 * gemm_ff.h -- C ABI of libttcff: the feed-forward part of a model on NVIDIA B200
 * (sm_100a), beside libttc05 (gemm_f16.h) and libttcmx (gemm_mx.h), whose status
 * codes, activations, 16-bit types and stream type it shares:
 *
 *   - the gated projections h = act(x Wg^T) * (x Wu^T) with 16-bit weights, one
 *     kernel from one token to long prompts, and their backward pass;
 *   - products of few rows with 4-bit weights that have a scale for each group of
 *     columns, plain and gated.
 *
 * Matrices are DEVICE pointers, 16-byte aligned, row-major; row strides are in
 * elements unless an entry point says otherwise and make rows start on 16 bytes
 * (a multiple of 8 elements of 16 bits, of 4 fp32 values, of 16 bytes).  Host
 * pointers and extents past the allocation are refused before any launch; calls
 * are asynchronous and stream-ordered; results are the same bits on every run on one
 * GPU (into how many parts a sum is divided depends on the sizes and on how many
 * clusters the GPU holds); errors found on the device are read with
 * ff_get_device_status().  No entry point throws, allocates device memory or keeps a
 * reference to its arguments, so calls on several streams or host threads share nothing, and every call can be captured
 * in a CUDA graph (make one such call outside a capture first: it looks up the
 * device and sets up the kernels).  Outputs must not overlap inputs or each other.
 *
 * Activations: gemm_activation (GEMM_ACT_NONE, _RELU, _GELU) and FF_ACT_SILU,
 * x / (1 + exp(-x)).  GELU is x Phi(x).  ReLU maps NaN to +0.
 */
#ifndef TTCFF_GEMM_FF_H
#define TTCFF_GEMM_FF_H

#include "gemm_mx.h"

#ifdef __cplusplus
extern "C" {
#endif

enum ff_activation { FF_ACT_SILU = 3 };

/* H = act(X Wg^T) * (X Wu^T).
 *   X: M x D, Wg, Wu: F x D, H: M x F, of type `dtype` (MX_F16 or MX_BF16);
 *   G, U: M x F fp32, the two projections before the activation, for
 *         ff_gated_backward; both or neither (NULL).
 * Sums and everything up to H's one rounding are fp32.  Sizes in [0, 2^31 - 256];
 * without rows or without columns F a no-op; D == 0 gives zeros. */
GEMM_API int ff_gated(const void* X, const void* Wg, const void* Wu, void* H, void* G, void* U,
                      int64_t M, int64_t F, int64_t D, int64_t ldx, int64_t ldwg, int64_t ldwu,
                      int64_t ldh, int64_t ldg, int64_t ldu, int dtype, int activation,
                      gemm_stream_t stream);

/* The backward pass, from the gradient dH of H and what ff_gated has left in G and U:
 *   dG = dH * U * act'(G),  dU = dH * act(G)
 *   dX  = dG Wg + dU Wu                   (NULL: not computed)
 *   dWg = dG^T X,  dWu = dU^T X           (both or neither NULL)
 * dG and dU (M x F, type dtype) are written by every call: each is rounded once, for
 * the tensor cores; everything before is fp32, as are the sums.  (In fp16 a dG or dU of
 * more than 65504 in magnitude is infinite there and one below 2^-25 zero: scale dH, as
 * is usual with fp16 gradients, or take bf16.)  act'(0) is 0 for ReLU.  With F == 0 dX is zeros, with M == 0 dWg and dWu are. */
GEMM_API int ff_gated_backward(const void* dH, const void* X, const void* Wg, const void* Wu,
                               const void* G, const void* U, void* dG, void* dU, void* dX,
                               void* dWg, void* dWu, int64_t M, int64_t F, int64_t D,
                               int64_t lddh, int64_t ldx, int64_t ldwg, int64_t ldwu, int64_t ldg,
                               int64_t ldu, int64_t lddg, int64_t lddu, int64_t lddx,
                               int64_t lddwg, int64_t lddwu, int dtype, int activation,
                               gemm_stream_t stream);

/* A 4-bit weight W of N x K in groups of 32, 64 or 128 columns,
 *   W[n][k] = (code[n][k] - zero[k / group][n]) * scale[k / group][n]:
 *   Q: codes 0 .. 15, row stride ldq in BYTES (a multiple of 16, >= K / 2 rounded
 *      up to 4).  Each 32-bit word (little endian) holds 8 consecutive columns:
 *      column 2 i of them in bits 4 i .. 4 i + 3, column 2 i + 1 in bits
 *      4 i + 16 .. 4 i + 19 (i = 0 .. 3), so that two neighbours come out of a word
 *      with one mask.  Columns past K may hold anything.
 *   S: scales, (K / group rounded up) x N, of the products' 16-bit type;
 *   Z: zero points 0 .. 15, (K / group rounded up) x N bytes, row stride ldz in
 *      bytes (a multiple of 16), or NULL: 8 for all.
 *
 * Y = act(X W^T + bias).  X: M x K, Y: M x N, bias: N values or NULL, of type dtype.
 * Codes and zero points are exact, the sums of a group are fp32 and take its scale
 * there: no weight is rounded.  (With up to 8 rows a group's codes and its zero point
 * are summed apart, so that an fp32 sum's error counts code + zero, not their
 * difference, and x is held to 2^-35 of the largest value of its row in the group.)  Made
 * for few rows: a weight is read once for every 64 of them.  K == 0 gives act(bias). */
GEMM_API int ff_w4_gemm(const void* X, const void* Q, const void* S, const void* Z,
                        const void* bias, void* Y, int64_t M, int64_t N, int64_t K, int64_t ldx,
                        int64_t ldq, int64_t lds, int64_t ldz, int64_t ldy, int group, int dtype,
                        int activation, gemm_stream_t stream);

/* H = act(X Wg^T) * (X Wu^T) with two such weights of F x D and one group size. */
GEMM_API int ff_w4_gated(const void* X, const void* Qg, const void* Sg, const void* Zg,
                         const void* Qu, const void* Su, const void* Zu, void* H, int64_t M,
                         int64_t F, int64_t D, int64_t ldx, int64_t ldqg, int64_t ldsg,
                         int64_t ldzg, int64_t ldqu, int64_t ldsu, int64_t ldzu, int64_t ldh,
                         int group, int dtype, int activation, gemm_stream_t stream);

/* Synchronises `stream`, then reports and clears this library's status word of the
 * current device, as gemm_get_device_status does for libttc05's. */
GEMM_API int ff_get_device_status(gemm_stream_t stream, int* device_status);

GEMM_API int ff_abi_version(void); /* 10000 */

#ifdef __cplusplus
}
#endif

#endif /* TTCFF_GEMM_FF_H */
