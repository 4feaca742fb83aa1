// 4-bit codes to 16-bit operands, exact, for the products with 4-bit weights.
#pragma once

#include "ff_common.cuh"

namespace ttc {
namespace ff {

// A zero point as what dequantize8 subtracts, twice in a word: of 1024 + code (fp16)
// or 128 + code (bf16), the numbers whose last mantissa bits are the code.
template <class T>
__device__ __forceinline__ uint32_t zero_pair(uint32_t z) {
  return (z | (std::is_same<T, __half>::value ? 0x6400u : 0x4300u)) * 0x10001u;
}

// The 8 codes of a word minus the zero point, in pairs of neighbours.
template <class T>
__device__ __forceinline__ void dequantize8(uint32_t w, uint32_t zero, uint32_t* p) {
  if constexpr (std::is_same<T, __half>::value) {
    // bits 4 .. 7 of a half hold 16 times the code: 1024 + 16 code, divided by 16
    // and minus 64 + zero in one fused step (all exact)
    const __half2 z = *reinterpret_cast<const __half2*>(&zero);
    const __half2 sixteenth = __float2half2_rn(0.0625f);
    const __half2 z64 = __hsub2(__float2half2_rn(960.0f), z);  // -(64 + zero)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t v = w >> (8 * i);
      const uint32_t lo = (v & 0x000F000Fu) | 0x64006400u, hi = (v & 0x00F000F0u) | 0x64006400u;
      const __half2 a = __hsub2(*reinterpret_cast<const __half2*>(&lo), z);
      const __half2 b = __hfma2(*reinterpret_cast<const __half2*>(&hi), sixteenth, z64);
      p[2 * i] = *reinterpret_cast<const uint32_t*>(&a);
      p[2 * i + 1] = *reinterpret_cast<const uint32_t*>(&b);
    }
  } else {
    const __nv_bfloat162 z = *reinterpret_cast<const __nv_bfloat162*>(&zero);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t v = ((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
      const __nv_bfloat162 a = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v), z);
      p[i] = *reinterpret_cast<const uint32_t*>(&a);
    }
  }
}

}  // namespace ff
}  // namespace ttc
