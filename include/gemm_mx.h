/*
 * gemm_mx.h -- C ABI of libttcmx: microscaled (MX) operands for the products
 * of a linear layer on NVIDIA B200 (sm_100a), the companion of libttc05
 * (gemm_f16.h, whose status codes, activations and stream type it shares).
 *
 * An MX matrix holds 8- or 4-bit floating-point elements with one power-of-two
 * scale for each block of 32 consecutive elements of a row, as defined by the
 * OCP Microscaling Formats (MX) Specification v1.0 (sections 5 and 6.3):
 *
 *   block maximum m  ->  e = floor(log2 m) - emax,  clamped to [-127, 127]
 *   scale            ->  X = 2^e, stored as the byte e + 127 (E8M0)
 *   element          ->  x / X rounded to nearest even, saturating
 *
 *   MX_FP8: E4M3 elements (emax 8, largest 448), one byte each;
 *   MX_FP4: E2M1 elements (emax 2, largest 6), two to a byte, the element
 *           with the even index in the low half.
 *
 *   - A block of zeros has scale byte 0.  A block that holds a NaN or an
 *     infinity has scale byte 255 (NaN) and zero elements: everything in it
 *     stands for NaN, and so do the outputs of a product that read it.
 *   - The last block of a row may be short: what is missing counts as zero.
 *
 * Storage of an MX matrix of rows x cols
 *   - data: one row after the other, `ld` BYTES apart, ld a multiple of 16 and
 *     >= mx_row_bytes(cols, format); 16-byte aligned.  With MX_FP4 and odd
 *     cols the last byte of a row has 0 in its high half.  Bytes of a row
 *     past mx_row_bytes are neither read nor written.
 *   - scales: mx_scale_bytes(rows, cols) bytes, 16-byte aligned: one tile of
 *     512 bytes for each 128 rows and each 128 columns (4 blocks), in the
 *     order the tensor cores take them.  The scale of row r and block b is
 *     byte (r % 32) * 16 + (r % 128 / 32) * 4 + b % 4 of tile
 *     (r / 128) * ceil(cols / 128) + b / 4.  Places without a row or a block
 *     hold 0: mx_quantize and mx_rms_norm write them so, and a matrix built in
 *     another way must hold no 255 in the places past its last block.
 *
 * 16-bit matrices (inputs, outputs, bias) are IEEE binary16 (MX_F16) or
 * bfloat16 (MX_BF16).  As in gemm_f16.h they are DEVICE pointers, 16-byte
 * aligned, row-major with row strides in elements that are multiples of 8;
 * host pointers and extents past the allocation are refused before any
 * launch; calls are asynchronous and stream-ordered; results are the same bits
 * on every run; errors found on the device are read with
 * mx_get_device_status().  No entry point throws, allocates device memory or
 * keeps a reference to its arguments, so calls on several streams or host
 * threads share nothing, and every call can be captured in a CUDA graph (make
 * one such call outside a capture first: it looks up the device and sets up the
 * kernel).  Outputs must
 * not overlap inputs unless an entry point says so.
 */
#ifndef TTCMX_GEMM_MX_H
#define TTCMX_GEMM_MX_H

#include "gemm_f16.h"

#ifdef __cplusplus
extern "C" {
#endif

enum mx_format {
  MX_NONE = 0, /* mx_rms_norm: 16-bit output */
  MX_FP8 = 1,  /* E4M3 elements, block of 32, E8M0 scale */
  MX_FP4 = 2   /* E2M1 elements, block of 32, E8M0 scale */
};

enum mx_dtype { MX_F16 = 0, MX_BF16 = 1 };

/* Bytes of a row of `cols` elements, and of the scales of a rows x cols
 * matrix; -1 for a bad format or a negative size. */
GEMM_API int64_t mx_row_bytes(int64_t cols, int format);
GEMM_API int64_t mx_scale_bytes(int64_t rows, int64_t cols);

/* (Q, S) = MX of X.  X: rows x cols, 16-bit of type `dtype`, row stride ldx
 * (elements).  Q: row stride ldq (bytes).  Sizes in [0, 2^31 - 1]; a matrix
 * without rows or columns is a no-op.  Exact: every element is the correctly
 * rounded quotient. */
GEMM_API int mx_quantize(const void* X, void* Q, void* S, int64_t rows, int64_t cols, int64_t ldx,
                         int64_t ldq, int dtype, int format, gemm_stream_t stream);

/* X = the values that (Q, S) stands for, rounded to `dtype` (a value outside
 * the range of binary16 becomes an infinity or a subnormal, as in any
 * conversion). */
GEMM_API int mx_dequantize(const void* Q, const void* S, void* X, int64_t rows, int64_t cols,
                           int64_t ldq, int64_t ldx, int dtype, int format,
                           gemm_stream_t stream);

/* The root-mean-square norm of each row, optionally of a residual sum and
 * optionally straight to MX:
 *   h = X                          (R == NULL)
 *   h = X + R rounded to `dtype`   (R != NULL), stored to H unless H is NULL
 *   y = h / sqrt(mean(h^2) + eps) * W
 *   format MX_NONE: Y = y rounded to `dtype`, row stride ldy in elements;
 *                   S is ignored
 *   MX_FP8 / MX_FP4: (Y, S) = MX of y, row stride ldy in bytes, without a
 *                   rounding in between
 * X, R, H: rows x cols of type dtype, W: cols values of type dtype, 16-byte
 * aligned.  H may be X or R itself (the stream updated in place), and Y with
 * MX_NONE may be X itself when R is NULL.  The mean is taken over the exact
 * squares; every output is y correctly rounded (to about 2^-43 beside a tie).
 * (h * W is held in fp32, with h times 2^80 or 2^-80 in rows whose squares leave
 * fp32's range: so scaled, |h * W| up to 3e38, and from about 1e-31 for that
 * precision.)  eps >= 0. */
GEMM_API int mx_rms_norm(const void* X, const void* R, const void* W, void* H, void* Y, void* S,
                         int64_t rows, int64_t cols, int64_t ldx, int64_t ldr, int64_t ldh,
                         int64_t ldy, float eps, int dtype, int format, gemm_stream_t stream);

/* C = act(A @ B^T + bias).
 *   A: M x K MX matrix (data A, row stride lda in bytes, scales SA);
 *   B: N x K MX matrix of the same format (the weight of a linear layer);
 *   bias: N values of type `dtype`, 16-byte aligned, or NULL;
 *   C: M x N of type `dtype`, row stride ldc in elements;
 *   activation: a gemm_activation value.
 * Products and sums are fp32; C is rounded once.  K == 0 gives C = act(bias).
 * GELU is x Phi(x), before the rounding right to 2^-18 + x^2 2^-22 relative, down
 * its negative tail, too (NaN for -infinity).
 * An output whose row of A or of B holds a NaN block is NaN (+0 after ReLU,
 * which maps NaN to +0). */
GEMM_API int mx_gemm(const void* A, const void* SA, const void* B, const void* SB,
                     const void* bias, void* C, int64_t M, int64_t N, int64_t K, int64_t lda,
                     int64_t ldb, int64_t ldc, int format, int dtype, int activation,
                     gemm_stream_t stream);

/* Synchronises `stream`, then reports and clears this library's status word
 * of the current device, as gemm_get_device_status does for libttc05's. */
GEMM_API int mx_get_device_status(gemm_stream_t stream, int* device_status);

GEMM_API int mx_abi_version(void); /* 10000 */

#ifdef __cplusplus
}
#endif

#endif /* TTCMX_GEMM_MX_H */
