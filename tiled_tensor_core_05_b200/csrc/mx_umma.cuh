// tcgen05 helpers of the MX products (block-scaled MMA, scale factors in
// TMEM), in the manner of sm100.cuh.
//
// An operand stage is 128 bytes of each row (128 E4M3 or 256 E2M1 elements) in
// the 128-byte-swizzled K-major layout, and the matching scale tiles (one of
// 512 bytes per 128 elements and 128 rows) as they lie in memory.  One MMA
// takes 32 bytes of K: 32 E4M3 elements = one scale a row, or 64 E2M1
// elements = two.
#pragma once

#include <type_traits>

#include "mx_common.cuh"
#include "mx_internal.h"

namespace ttc {
namespace mx {

template <int FMT>
struct Kind {
  static constexpr int kStageK = FMT == MX_FP8 ? 128 : 256;  // elements per stage
  static constexpr int kSfTiles = FMT == MX_FP8 ? 1 : 2;     // scale tiles per stage
  static constexpr int kSfCols = 4 * kSfTiles;               // TMEM columns of a stage's scales
};
constexpr int kRowBytes = 128;  // bytes of a row in a stage
constexpr int kMmaBytes = 32;   // bytes of a row that one MMA takes
constexpr int kMmasPerStage = kRowBytes / kMmaBytes;

// Instruction descriptor of the block-scaled kinds.
//   bits 4-5 scale-factor id of B, 7-9 A format, 10-12 B format, 17-22 N >> 3,
//   23 scale type (1 = UE8M0), 27-28 M >> 7, 29-30 scale-factor id of A;
//   A and B K-major.  E4M3 is 0 of kind::mxf8f6f4, E2M1 is 1 of kind::mxf4.
// The scale-factor id names the byte of each 32-bit scale word to start from.
template <int FMT>
__host__ __device__ constexpr uint32_t mx_idesc(int m, int n, int k) {
  const uint32_t f = FMT == MX_FP8 ? 0u : 1u;
  const uint32_t id = FMT == MX_FP8 ? static_cast<uint32_t>(k) : 2u * static_cast<uint32_t>(k & 1);
  return (id << 4) | (f << 7) | (f << 10) | (static_cast<uint32_t>(n >> 3) << 17) | (1u << 23) |
         (static_cast<uint32_t>(m >> 7) << 27) | (id << 29);
}

// The MMA warp runs its loop as a whole, so that descriptors and addresses stay
// in uniform registers (a lane of its own would move every operand of every
// instruction there: 225 instead of 204 us at 8192 x 14336 x 4096 MXFP4); one
// elected lane issues.  So does the producer warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ bool mbar_wait_warp(uint64_t* bar, uint32_t parity,
                                               const volatile int* abort_flag,
                                               uint64_t timeout_ns) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, timeout_ns)) != 0;
}

// Descriptors: an operand's rows of 128 bytes, 128-byte swizzled, K-major
// (smem_desc_sw128); a scale tile's 32 rows of 16 bytes, no swizzle, 8-row
// groups 128 bytes apart.
//
// One thread issues all of this, and its instructions are what a k-block's
// time comes down to, so descriptors are two 32-bit words of which only the
// low one changes (address >> 4; nothing carries out of it), and what can be
// is a constant.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
constexpr uint32_t kScaleDescHigh = (128u >> 4) | (1u << 14);
__device__ __forceinline__ uint32_t desc_low(uint32_t saddr) { return (saddr >> 4) | (1u << 16); }

// A scale tile from shared memory (address >> 4) to 4 TMEM columns, repeated in
// the four 32-lane quarters: lane l, column c holds the scales of row 32 c + l.
template <int CTAS>
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint32_t low) {
  if constexpr (CTAS == 1)
    asm volatile(
        "{\n\t.reg .b64 d;\n\tmov.b64 d, {%1, %2};\n\t"
        "tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], d;\n\t}" ::"r"(taddr),
        "r"(low), "r"(kScaleDescHigh)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .b64 d;\n\tmov.b64 d, {%1, %2};\n\t"
        "tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], d;\n\t}" ::"r"(taddr),
        "r"(low), "r"(kScaleDescHigh)
        : "memory");
}

// D (+)= (A . SA) (B . SB), fp32 accumulator; a, b: low descriptor words.
#define TTC_MX_MMA(GROUP, KIND)                                                                   \
  asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tmov.b64 da, {%1, %7};\n\t"             \
               "mov.b64 db, {%2, %7};\n\tsetp.ne.b32 p, %6, 0;\n\t"                               \
               "tcgen05.mma.cta_group::" GROUP ".kind::" KIND " [%0], da, db, %3, [%4], [%5], p;" \
               "\n\t}\n" ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate),  \
               "r"(kDescHigh)                                                                     \
               : "memory")
template <int FMT, int CTAS>
__device__ __forceinline__ void mx_mma(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                       uint32_t sa, uint32_t sb, uint32_t accumulate) {
  if constexpr (FMT == MX_FP8 && CTAS == 1)
    TTC_MX_MMA("1", "mxf8f6f4.block_scale.scale_vec::1X");
  else if constexpr (FMT == MX_FP8)
    TTC_MX_MMA("2", "mxf8f6f4.block_scale.scale_vec::1X");
  else if constexpr (CTAS == 1)
    TTC_MX_MMA("1", "mxf4.block_scale.scale_vec::2X");
  else
    TTC_MX_MMA("2", "mxf4.block_scale.scale_vec::2X");
}
#undef TTC_MX_MMA

// The MMAs of one k-block into d: A of MMA shape M x N from a, B from b (shared
// addresses), scales of A from column sa and of B from sb on, 4 and
// SB_TILE columns per scale tile; `left` bytes of the row remain.
template <int FMT, int CTAS, int M, int N, int SB_TILE>
__device__ __forceinline__ void issue_mmas(uint32_t d, uint32_t a, uint32_t b, uint32_t sa,
                                           uint32_t sb, int left, bool accumulate) {
  const uint32_t al = desc_low(a), bl = desc_low(b);
  auto one = [&](auto k, uint32_t acc) {
    constexpr int K = decltype(k)::value;
    constexpr int t = FMT == MX_FP8 ? 0 : K / 2;
    mx_mma<FMT, CTAS>(d, al + K * (kMmaBytes >> 4), bl + K * (kMmaBytes >> 4),
                      mx_idesc<FMT>(M, N, K), sa + 4 * t, sb + SB_TILE * t, acc);
  };
  one(std::integral_constant<int, 0>{}, accumulate ? 1u : 0u);
  if (left >= kRowBytes) {
    one(std::integral_constant<int, 1>{}, 1u);
    one(std::integral_constant<int, 2>{}, 1u);
    one(std::integral_constant<int, 3>{}, 1u);
  } else {  // the last k-block: only the MMAs that reach into the row
    if (left > 1 * kMmaBytes) one(std::integral_constant<int, 1>{}, 1u);
    if (left > 2 * kMmaBytes) one(std::integral_constant<int, 2>{}, 1u);
    if (left > 3 * kMmaBytes) one(std::integral_constant<int, 3>{}, 1u);
  }
}

// Untiled copy of `bytes` (a multiple of 16) global -> shared, counted on `bar`.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// Copy of `bytes` (a multiple of 16) from this CTA's shared memory to that of
// another CTA of the cluster, counted on an mbarrier there (shared::cluster
// addresses).
__device__ __forceinline__ void bulk_push(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, "
      "[%3];" ::"r"(dst),
      "r"(smem_u32(src)), "r"(bytes), "r"(bar)
      : "memory");
}

// GELU(x) = x Phi(x) for outputs that are rounded relative to their size far
// down the negative tail (in bf16 to x = -13), where the form of sm100.cuh,
// whose Phi is right to an absolute 0.75e-7, is off by 0.05 % at x = -4, 0.2 % at
// -5.5 and 2 % at -10.  Here
//   Phi(-|x|) = exp(-z^2) (c1 t + c2 t^2 + ... + c7 t^7),  z = |x| / sqrt 2,
//   t = 1 / (1 + p z),  p = 0.3725,
// a minimax fit to erfc(z) exp(z^2) / 2 in relative terms over 0 <= z <= 9.6
// (linear programming on 1500 Chebyshev points of t, p by search): 5.4e-7.
// With the fp32 roundings, above all of z in the exponent, the value is right
// to 2^-18 + x^2 2^-22 relative.
//
// In the variable u = z sqrt(log2 e) = kU |x|: GELU = max(x, 0) - |x| Phi(-|x|) =
// max(x, 0) + u T with -1 / kU in T's coefficients, two values at a time.  The
// exponent is 8 - u^2 and 2^-8 in the coefficients, too, so that 2^(8 - u^2), where
// the instruction flushes what is subnormal, is lost only where the result is
// below half of bf16's smallest value.  u comes from min(x, 2^100): infinity gives
// infinity, -infinity NaN as 0 times -infinity does, and NaN stays NaN.
//
// Seven terms and this form take as many instructions as five terms and a
// selection of Phi(x) or 1 - Phi(-x): 8192 x 14336 x 4096 MXFP4 with bias 190.5 us
// in both types, 192.5 with the form of sm100.cuh.
constexpr float kGeluU = 0.8493218002880191f;   // sqrt(1/2) sqrt(log2 e)
constexpr float kGeluP = 0.31012659265624243f;  // p / sqrt(log2 e)
constexpr float kGelu1 = 0.10492625832557678f;
constexpr float kGelu2 = 0.10768866539001465f;
constexpr float kGelu3 = 0.07959755510091782f;
constexpr float kGelu4 = 0.15073831379413605f;
constexpr float kGelu5 = -0.07991653680801392f;
constexpr float kGelu6 = 0.20664797723293304f;
constexpr float kGelu7 = -0.06968224048614502f;

__device__ __forceinline__ float2 gelu2_relative(float2 x) {
  constexpr float kC = static_cast<float>(-0x1p-8 / 0.8493218002880191);
  float2 v;
  asm("min.NaN.f32 %0, %1, 0f71800000;" : "=f"(v.x) : "f"(x.x));
  asm("min.NaN.f32 %0, %1, 0f71800000;" : "=f"(v.y) : "f"(x.y));
  const float2 u = __fmul2_rn(make_float2(fabsf(v.x), fabsf(v.y)), splat2(kGeluU));
  const float2 d = __ffma2_rn(u, splat2(kGeluP), splat2(1.0f));
  const float2 t = make_float2(rcp_approx(d.x), rcp_approx(d.y));
  float2 q = __ffma2_rn(splat2(kGelu7 * kC), t, splat2(kGelu6 * kC));
  q = __ffma2_rn(q, t, splat2(kGelu5 * kC));
  q = __ffma2_rn(q, t, splat2(kGelu4 * kC));
  q = __ffma2_rn(q, t, splat2(kGelu3 * kC));
  q = __ffma2_rn(q, t, splat2(kGelu2 * kC));
  q = __ffma2_rn(q, t, splat2(kGelu1 * kC));
  q = __fmul2_rn(q, t);
  const float2 w = __ffma2_rn(u, u, splat2(-8.0f));
  const float2 tail = __fmul2_rn(q, make_float2(ex2_approx(-w.x), ex2_approx(-w.y)));
  return __ffma2_rn(u, tail, make_float2(fmaxf(x.x, -0.0f), fmaxf(x.y, -0.0f)));
}

// The activations of the MX products.
template <int ACT>
__device__ __forceinline__ float2 mx_activate2(float2 x) {
  if constexpr (ACT == kActGelu)
    return gelu2_relative(x);
  else
    return activate2<ACT>(x);
}

// bias + activation in fp32 of two columns.
__device__ __forceinline__ float2 finish2(float2 v, float2 b, int act) {
  v = __fadd2_rn(v, b);
  return act == kActRelu   ? mx_activate2<kActRelu>(v)
         : act == kActGelu ? mx_activate2<kActGelu>(v)
                           : v;
}

// cluster_sync in two halves: every thread arrives once, then waits once.  The
// relaxed arrival orders nothing before it: it is for threads whose use of the
// others' shared memory has been seen to end (an mbarrier they waited for).
// A release waits for the thread's stores to global memory, too (some 1500
// cycles at the end of a kernel).
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_arrive_relaxed() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(r));
  return r;
}

__device__ __forceinline__ void add8(float (&v)[8], const float4& x, const float4& y) {
  v[0] += x.x, v[1] += x.y, v[2] += x.z, v[3] += x.w;
  v[4] += y.x, v[5] += y.y, v[6] += y.z, v[7] += y.w;
}

// Rows that a CTA has slots for in the kernels that divide K: of a tile of
// `rows` rows in n parts it finishes up to ceil(rows / n) and is sent them by the
// n - 1 others; the most over n <= max_parts (16 rows: 18 with 7 parts).
constexpr int slot_rows(int rows, int max_parts) {
  int most = 0;
  for (int n = 2; n <= max_parts; ++n) {
    const int r = (n - 1) * ((rows + n - 1) / n);
    most = r > most ? r : most;
  }
  return most;
}

// What the epilogues of the kernels that divide K need of C.
struct Output {
  uint16_t* C;
  const uint16_t* bias;
  int64_t ldc;
  int M, N;
  int dtype, act;
};

inline Output output_of(const MxGemmProblem& p) {
  return Output{static_cast<uint16_t*>(p.C), static_cast<const uint16_t*>(p.bias), p.ldc,
                static_cast<int>(p.M),       static_cast<int>(p.N),             p.dtype, p.act};
}

// The 8 columns from n on of some rows of C, n the same for all rows a thread
// finishes: what does not depend on the row is done once.
template <class T>
struct Columns {
  uint16_t* C;
  int64_t ldc;
  int count;
  float b[8];
  __device__ __forceinline__ Columns(const Output& o, int n, const uint4& bias)
      : C(o.C + n), ldc(o.ldc), count(min(8, o.N - n)) {
    unpack8<T>(bias, b);
  }
  // a row from its fp32 sums: bias, activation, one rounding, stored as 16
  // bytes or, across the edge, one by one
  template <int ACT>
  __device__ __forceinline__ void store(int m, const float (&v)[8]) const {
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const float2 r = mx_activate2<ACT>(
          __fadd2_rn(make_float2(v[i], v[i + 1]), make_float2(b[i], b[i + 1])));
      y[i] = r.x;
      y[i + 1] = r.y;
    }
    store8(C + static_cast<int64_t>(m) * ldc, pack8<T>(y), count);
  }
};

// The bias of the columns from n on (0 without one), for Columns: loaded while
// the product's operands are still on their way.
__device__ __forceinline__ uint4 load_bias(const Output& o, int n) {
  if (o.bias == nullptr || n >= o.N) return make_uint4(0, 0, 0, 0);
  return load8(o.bias + n, min(8, o.N - n));
}

// f(columns, activation) with the type and the activation as constants: a row
// of the loop below is some 100 instructions, twice as many with them looked up
// each time, and the last rows of a tile have nothing to hide them behind.
template <class F>
__device__ __forceinline__ void with_columns(const Output& o, int n, const uint4& bias, F&& f) {
  auto typed = [&](auto columns) {
    if (o.act == kActRelu)
      f(columns, std::integral_constant<int, kActRelu>{});
    else if (o.act == kActGelu)
      f(columns, std::integral_constant<int, kActGelu>{});
    else
      f(columns, std::integral_constant<int, kActNone>{});
  };
  if (n >= o.N) return;
  if (o.dtype == MX_F16)
    typed(Columns<__half>(o, n, bias));
  else
    typed(Columns<__nv_bfloat16>(o, n, bias));
}

// Rows m of C (m counts from m0) as the sums of their parts, in the order of
// the parts; part(s) has the columns of this thread, 128 floats a row.  16
// threads a row.
template <int kThreads, class Part>
__device__ __forceinline__ void finish_rows(const Output& o, int m0, int n, int rows,
                                            const uint4& bias, int parts, Part&& part) {
  with_columns(o, n, bias, [&](const auto& columns, auto act) {
    for (int m = threadIdx.x >> 4; m < rows; m += kThreads / 16) {
      float v[8] = {};
      for (int s = 0; s < parts; ++s) {
        const float4* src = reinterpret_cast<const float4*>(part(s) + m * 128);
        add8(v, src[0], src[1]);
      }
      columns.template store<decltype(act)::value>(m0 + m, v);
    }
  });
}

}  // namespace mx
}  // namespace ttc
