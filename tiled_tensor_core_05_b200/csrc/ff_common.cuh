// Device helpers of the feed-forward operators: activations and their slopes,
// and the joining of sums that the CTAs of a cluster hold in parts.
#pragma once

#include "ff_internal.h"
#include "mx_umma.cuh"

namespace ttc {
namespace ff {

enum : int { kActSilu = FF_ACT_SILU };

// 1 / (1 + exp(-x)): 0 from where 2^126 is exceeded (x < -87.3) on, so that SiLU
// is lost only below 1e-36, and SiLU(-infinity) is NaN, as -infinity times 0 is.
__device__ __forceinline__ float sigmoid(float x) {
  return rcp_approx(1.0f + ex2_approx(-1.4426950408889634f * x));
}

template <int ACT>
__device__ __forceinline__ float2 ff_activate2(float2 x) {
  if constexpr (ACT == kActSilu)
    return __fmul2_rn(x, make_float2(sigmoid(x.x), sigmoid(x.y)));
  else
    return mx::mx_activate2<ACT>(x);
}

// act(x) and act'(x).
//   SiLU:  p = sigmoid(x); x p and p (1 + x (1 - p))
//   GELU:  x Phi(x) and Phi(x) + x phi(x), with Phi(-|x|) = exp(-x^2 / 2) times the
//          polynomial of mx::gelu2_relative, whose exponential phi shares
//   ReLU:  slope 0 at 0
template <int ACT>
__device__ __forceinline__ void value_and_slope(float x, float& value, float& slope) {
  if constexpr (ACT == kActSilu) {
    const float p = sigmoid(x);
    value = x * p;
    slope = fmaf(value, 1.0f - p, p);
  } else if constexpr (ACT == kActGelu) {
    const float u = fabsf(x) * mx::kGeluU;
    const float t = rcp_approx(fmaf(u, mx::kGeluP, 1.0f));
    float q = fmaf(mx::kGelu7, t, mx::kGelu6);
    q = fmaf(q, t, mx::kGelu5);
    q = fmaf(q, t, mx::kGelu4);
    q = fmaf(q, t, mx::kGelu3);
    q = fmaf(q, t, mx::kGelu2);
    q = fmaf(q, t, mx::kGelu1);
    const float e = ex2_approx(-u * u);  // exp(-x^2 / 2)
    const float tail = q * t * e;
    const float phi = x < 0.0f ? tail : 1.0f - tail;
    value = x * phi;
    slope = fmaf(x * e, 0.3989422804014327f, phi);
  } else if constexpr (ACT == kActRelu) {
    value = relu_f32(x);
    slope = x > 0.0f ? 1.0f : 0.0f;
  } else {
    value = x;
    slope = 1.0f;
  }
}

// f(integral_constant) for the activation code.
template <class F>
__device__ __forceinline__ void with_act(int act, F&& f) {
  if (act == kActSilu)
    f(std::integral_constant<int, kActSilu>{});
  else if (act == kActGelu)
    f(std::integral_constant<int, kActGelu>{});
  else if (act == kActRelu)
    f(std::integral_constant<int, kActRelu>{});
  else
    f(std::integral_constant<int, kActNone>{});
}

// ------------------------------------------------------------- sums in parts ---
// A kernel that divides K leaves each CTA of a cluster with a part of the tile's
// fp32 sums: rows of kPartCols values in its shared memory.  CTA r finishes the rows
// [rows r / n, rows (r + 1) / n): the others send it theirs (one bulk copy between
// the SMs' shared memories each) and it adds the parts in rank order; their number
// depends on the shape and on how many clusters the GPU holds.  Up to kPullRows rows the first CTA reads the others' parts
// instead: copies would take longer than the loads.
constexpr int kPartCols = 128;
constexpr int kMaxSplits = 8;  // CTAs of a cluster
constexpr int kPullRows = 4;

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// What the last rows of a tile need.
struct Tail {
  uint16_t* Y;
  const uint16_t* bias;  // plain products only
  float *gate, *up;      // gated products only; may be null
  int64_t ldy, ld_gate, ld_up;
  int M, N;  // rows and columns of Y
  int dtype, act;
  int gated;
};

__device__ __forceinline__ void store_f32x8(float* p, const float (&v)[8], int n) {
  if (n >= 8) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = v[i];
  }
}

// Finishes rows m0 .. m0 + rows - 1 of Y; sum(m, v) gives the 8 sums of the part
// column 8 (threadIdx.x % 16) of row m0 + m.  16 threads a row.  Plain: part column
// c is column n0 + c of Y.  Gated: part columns 0 .. 63 are the gate's and 64 .. 127
// the other projection's columns n0 .. n0 + 63: the lower 8 threads of a row take
// the upper 8's sums.
template <int kThreads, class Sum>
__device__ __forceinline__ void finish_rows(const Tail& o, int m0, int n0, int rows, Sum&& sum) {
  const int c = static_cast<int>(threadIdx.x & 15) * 8;
  auto typed = [&](auto type, auto act) {
    using T = decltype(type);
    constexpr int ACT = decltype(act)::value;
    const int n = n0 + (o.gated ? c & 63 : c);
    const int count = min(8, o.N - n);
    float b[8];
    uint4 raw = make_uint4(0, 0, 0, 0);
    if (o.bias != nullptr && count > 0) raw = mx::load8(o.bias + n, count);
    mx::unpack8<T>(raw, b);
    // (every lane of a warp takes part in the exchange)
    for (int base = 0; base < rows; base += kThreads / 16) {
      const int m = base + static_cast<int>(threadIdx.x >> 4);
      float v[8] = {}, y[8];
      if (m < rows) sum(m, v);
      if (o.gated) {
        float u[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = __shfl_down_sync(0xffffffffu, v[i], 8, 16);
        if (c >= 64 || m >= rows || count <= 0) continue;
        if (o.gate != nullptr) {
          store_f32x8(o.gate + (m0 + m) * o.ld_gate + n, v, count);
          store_f32x8(o.up + (m0 + m) * o.ld_up + n, u, count);
        }
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const float2 r = __fmul2_rn(ff_activate2<ACT>(make_float2(v[i], v[i + 1])),
                                      make_float2(u[i], u[i + 1]));
          y[i] = r.x;
          y[i + 1] = r.y;
        }
      } else {
        if (m >= rows || count <= 0) continue;
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const float2 r = ff_activate2<ACT>(
              __fadd2_rn(make_float2(v[i], v[i + 1]), make_float2(b[i], b[i + 1])));
          y[i] = r.x;
          y[i + 1] = r.y;
        }
      }
      mx::store8(o.Y + (m0 + m) * o.ldy + n, mx::pack8<T>(y), count);
    }
  };
  with_act(o.act, [&](auto act) {
    if (o.dtype == MX_F16)
      typed(__half{}, act);
    else
      typed(__nv_bfloat16{}, act);
  });
}

// Joins and finishes a tile of `rows` rows whose part lies at `part` (row stride
// kPartCols values), with room for what others send behind it.  Every thread has
// arrived once at the cluster's barrier (splits > 1): with up to kPullRows rows released,
// after it has written its share of the part; with more, once it reads and writes
// nothing any more of the ring that the incoming parts overwrite.
// kThreads threads, all of them here; afterwards no CTA reads or signals another.
template <int BN, int kThreads>
__device__ __forceinline__ void join_and_finish(const Tail& o, uint8_t* part, uint64_t* received,
                                                volatile int* abort_flag, int* status,
                                                uint64_t timeout_ns, int rank, int splits, int m0,
                                                int n0, int rows) {
  auto first_row = [&](int r) { return rows * r / splits; };
  const int r0 = first_row(rank), r1 = first_row(rank + 1);
  const int slot_bytes = (BN + splits - 1) / splits * kPartCols * 4;
  const bool pull = rows <= kPullRows;
  uint8_t* incoming = part + BN * kPartCols * 4;
  const int c = static_cast<int>(threadIdx.x & 15) * 8;
  if (splits > 1) {
    fence_proxy_async_smem();  // the part is read by bulk copies
    __syncthreads();           // all of this CTA's part is written
    mx::cluster_wait();        // pull: all parts are; push: all rings are free
    if (!pull && threadIdx.x == 0) {
      mbar_arrive_expect_tx(received,
                            static_cast<uint32_t>((splits - 1) * (r1 - r0) * kPartCols * 4));
      for (int k = 1; k < splits && *abort_flag == 0; ++k) {
        const int to = rank + k < splits ? rank + k : rank + k - splits;
        const int from_row = first_row(to), n = first_row(to + 1) - from_row;
        if (n == 0) continue;
        // the receiver keeps its slots in rank order, without its own
        const int slot = rank < to ? rank : rank - 1;
        mx::bulk_push(map_to_cta(smem_u32(incoming) + static_cast<uint32_t>(slot * slot_bytes),
                                 static_cast<uint32_t>(to)),
                      part + from_row * kPartCols * 4, static_cast<uint32_t>(n * kPartCols * 4),
                      map_to_cta(smem_u32(received), static_cast<uint32_t>(to)));
      }
    }
    // (after an abort, too: what others have sent has to land before this CTA ends)
    if (!pull && r1 > r0 && !mbar_wait(received, 0, nullptr, timeout_ns))
      raise_abort(status, abort_flag, kStatusTimeoutBase | (kRoleEpilogue << 4) | 2);
  } else {
    __syncthreads();
  }
  // One answer a warp where finish_rows exchanges sums between its lanes: a wait that runs out
  // may have ended well for some of them.  (Asked by all calls, the compiler makes a function of
  // finish_rows: 1000 x 1000 -> 1000 15.1 us instead of 14.2.)
  bool aborted = *abort_flag != 0;
  if (splits > 1 && o.gated) aborted = __any_sync(0xffffffffu, aborted);
  if (splits > 1 && pull) {
    static_assert(kPullRows * 16 <= kThreads, "a row for 16 threads");
    float v[8] = {};
    const int m = static_cast<int>(threadIdx.x >> 4);
    if (rank == 0 && m < rows) {
      float4 p[kMaxSplits][2];  // all parts are on their way before the first is added
#pragma unroll
      for (int s = 0; s < kMaxSplits; ++s) {
        if (s >= splits) break;
        const uint32_t src =
            map_to_cta(smem_u32(part) + static_cast<uint32_t>(m * kPartCols + c) * 4,
                       static_cast<uint32_t>(s));
        p[s][0] = ld_cluster_f4(src);
        p[s][1] = ld_cluster_f4(src + 16);
      }
#pragma unroll
      for (int s = 0; s < kMaxSplits; ++s) {
        if (s >= splits) break;
        mx::add8(v, p[s][0], p[s][1]);
      }
    }
    __syncwarp();
    // the others' parts have been read: their owners may leave
    if (rank == 0)
      mx::cluster_arrive();
    else
      mx::cluster_arrive_relaxed();
    if (rank == 0 && !aborted)
      finish_rows<kThreads>(o, m0, n0, rows, [&](int, float(&s)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] = v[i];
      });
  } else {
    __syncwarp();
    if (splits > 1) mx::cluster_arrive_relaxed();  // what was sent here has left the others
    if (!aborted)
      finish_rows<kThreads>(o, m0 + r0, n0, r1 - r0, [&](int m, float(&v)[8]) {
        for (int s = 0; s < splits; ++s) {
          const uint8_t* rows_of =
              s == rank ? part + r0 * kPartCols * 4
                        : incoming + (s < rank ? s : s - 1) * slot_bytes;
          const float4* src =
              reinterpret_cast<const float4*>(reinterpret_cast<const float*>(rows_of) +
                                              m * kPartCols + c);
          mx::add8(v, src[0], src[1]);
        }
      });
  }
  __syncwarp();
  // no CTA leaves while another, or its own copies, may still read its shared memory
  if (splits > 1)
    mx::cluster_wait();
  else
    __syncthreads();
}

}  // namespace ff
}  // namespace ttc
