// Device helpers of the microscaled (MX) operators: 16-bit loads and stores,
// the conversion of a block to E4M3 / E2M1 elements and an E8M0 scale, and the
// layout of the scales.
//
// OCP Microscaling Formats (MX) Specification v1.0, sections 5 and 6.3: 32
// consecutive elements share X = 2^e, e = floor(log2(max |x|)) - emax; an
// element is x / X rounded to nearest even, saturating.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "../../include/gemm_mx.h"
#include "sm100.cuh"

namespace ttc {
namespace mx {

constexpr int kTileRows = 128;   // rows of a scale tile
constexpr int kTileCols = 128;   // columns of a scale tile (4 blocks)
constexpr int kTileBytes = 512;

// ---------------------------------------------------------------- 16-bit types ---
template <class T>
__device__ __forceinline__ float2 unpack2(uint32_t v);
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t v) {
  return __half22float2(*reinterpret_cast<const __half2*>(&v));
}
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t v) {
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}

template <class T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  return pack_half2(lo, hi);
}
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
  __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}

// Eight 16-bit elements at p, of which the first n exist (the others read as
// +0 and are not touched).
__device__ __forceinline__ uint4 load8(const uint16_t* p, int n) {
  if (n >= 8) return *reinterpret_cast<const uint4*>(p);
  uint4 v = make_uint4(0, 0, 0, 0);
  uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) w[i >> 1] |= static_cast<uint32_t>(p[i]) << (16 * (i & 1));
  return v;
}

__device__ __forceinline__ void store8(uint16_t* p, const uint4& v, int n) {
  if (n >= 8) {
    *reinterpret_cast<uint4*>(p) = v;
    return;
  }
  const uint32_t* w = reinterpret_cast<const uint32_t*>(&v);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) p[i] = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
}

template <class T>
__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(&v);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = unpack2<T>(w[i]);
    f[2 * i] = x.x;
    f[2 * i + 1] = x.y;
  }
}

template <class T>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]), pack2<T>(f[4], f[5]),
                    pack2<T>(f[6], f[7]));
}

// ------------------------------------------------------------------- elements ---
// Two values to two E4M3 bytes / four to two E2M1 bytes, round to nearest
// even, saturating; the first value lowest.
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}

__device__ __forceinline__ uint32_t e2m1x8(const float (&f)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
  return r;
}

// The other way, exact: two E4M3 bytes / eight E2M1 half bytes to fp32.
__device__ __forceinline__ float2 from_e4m3x2(uint32_t v) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(v)));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

__device__ __forceinline__ void from_e2m1x8(uint32_t v, float (&f)[8]) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(v));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    f[2 * i] = x.x;
    f[2 * i + 1] = x.y;
  }
}

// --------------------------------------------------------------------- scales ---
template <int FMT>
constexpr int kEmax = FMT == MX_FP8 ? 8 : 2;

// The scale byte of a block whose largest |x| has the fp32 bits `amax`
// (compared as integers, so a NaN or an infinity wins).  The exponent field
// is floor(log2) + 127; a subnormal maximum (field 0) clamps to byte 0 like
// every exponent below -127.
template <int FMT>
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
  const int field = static_cast<int>(amax >> 23);
  return field == 255 ? 255u : static_cast<uint32_t>(max(field - kEmax<FMT>, 0));
}

// 1 / X for a finite scale byte (at most 252 by construction: field >= 2).
__device__ __forceinline__ float inverse_scale(uint32_t byte) {
  return __uint_as_float((254u - byte) << 23);
}

// X; byte 0 is the subnormal 2^-127, byte 255 is NaN.
__device__ __forceinline__ float scale_value(uint32_t byte) {
  return byte == 255u ? __uint_as_float(0x7FC00000u)
                      : __uint_as_float(byte == 0u ? 0x00400000u : byte << 23);
}

__host__ __device__ __forceinline__ int64_t scale_tiles(int64_t cols) {
  return (cols + kTileCols - 1) / kTileCols;
}

// Byte offset of the 4 scales of row r, columns 128 kt .. 128 kt + 127.
__device__ __forceinline__ int64_t scale_word(int64_t r, int64_t kt, int64_t tiles) {
  return ((r >> 7) * tiles + kt) * kTileBytes + (r & 31) * 16 + ((r >> 5) & 3) * 4;
}

// max(|a|, |b|, |c|); NaN (0x7FFFFFFF) if one is NaN.
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)), "f"(fabsf(c)));
  return r;
}

// The MX form of 8 values of a row, a quarter of a block: called by all lanes
// of a warp, 4 consecutive lanes holding the values of a block (missing ones
// as 0).  Returns the block's scale byte; `q` receives the elements: 2 words
// of E4M3 or 1 of E2M1.
template <int FMT>
__device__ __forceinline__ uint32_t quantize8(const float (&y)[8], uint32_t (&q)[2]) {
  uint32_t amax = __float_as_uint(max3_abs(max3_abs(max3_abs(y[0], y[1], y[2]), y[3], y[4]),
                                           max3_abs(y[5], y[6], y[7]), 0.0f));
  amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  const uint32_t byte = scale_byte<FMT>(amax);
  q[0] = q[1] = 0;
  if (byte != 255u) {
    const float inv = inverse_scale(byte);  // a power of two: the products are exact
    float z[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = y[i] * inv;
    if constexpr (FMT == MX_FP8) {
      q[0] = e4m3x2(z[0], z[1]) | e4m3x2(z[2], z[3]) << 16;
      q[1] = e4m3x2(z[4], z[5]) | e4m3x2(z[6], z[7]) << 16;
    } else {
      q[0] = e2m1x8(z);
    }
  }
  return byte;
}

// Stores the elements of quantize8 at element column 8 i of a row's data, of
// which the first n exist.
template <int FMT>
__device__ __forceinline__ void store_elements(uint8_t* row, int64_t i, const uint32_t (&q)[2],
                                               int n) {
  if constexpr (FMT == MX_FP8) {
    uint8_t* p = row + 8 * i;
    if (n >= 8) {
      *reinterpret_cast<uint2*>(p) = make_uint2(q[0], q[1]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < n) p[j] = static_cast<uint8_t>(q[j >> 2] >> (8 * (j & 3)));
    }
  } else {
    uint8_t* p = row + 4 * i;
    if (n >= 7) {  // the 8th element is 0 where it does not exist
      *reinterpret_cast<uint32_t*>(p) = q[0];
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (2 * j < n) p[j] = static_cast<uint8_t>(q[0] >> (8 * j));
    }
  }
}

}  // namespace mx
}  // namespace ttc
