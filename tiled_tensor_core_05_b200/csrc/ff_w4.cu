// Products of few rows with 4-bit weights: act(X W^T + bias) and
// act(X Wg^T) * (X Wu^T), W = (code - zero) * scale in groups of GROUP columns.
//
// A tile is 128 rows of the weights (gated: 64 of the gate, the same 64 of the other
// projection) by BN rows of x; its K range is divided among the CTAs of a cluster
// and joined as in ff_common.cuh.  A stage of the ring is 256 columns: 128 bytes of
// each weight row, the rows of x, and the scales (and zero points) of its groups,
// all fetched by TMA, which fills what lies past N, M or K with zeros.
//
//   warp 8      TMA producer
//   warps 0-7   16 rows of the weights each: codes -> code - zero in 16 bits, exact,
//               in registers; mma.sync m16n8k16 with fp32 sums, from 0 for each group;
//               sums times scale added to the tile's in fp32
//
// The codes' fragments need no shuffle: the four threads that share a row of the MMA
// each take one 32-bit word (8 columns) of a 32-column chunk, and x's fragments the
// same 8 columns, which is the same sum in another order of K.
#include <atomic>

#include "ff_common.cuh"

namespace ttc {
namespace ff {
namespace {

constexpr int kWarps = 8;  // consumers
constexpr int kThreads = 32 * (kWarps + 1);
constexpr int kStageK = 256;                 // columns of a stage
constexpr int kChunks = kStageK / 32;
constexpr int kWBytes = kPartCols * kStageK / 2;
constexpr int kHalfRows = 64;                // rows of a weight box

template <int BN, int GROUP>
struct Cfg {
  static constexpr int kGroups = kStageK / GROUP;  // of a stage
  static constexpr int kXBytes = BN * kStageK * 2;
  static constexpr int kSBytes = kGroups * kPartCols * 2;
  static constexpr int kZBytes = kGroups * kPartCols;
  static constexpr int kStageBytes = kWBytes + kXBytes + kSBytes + kZBytes;
  static constexpr int kPartBytes = BN * kPartCols * 4;
  static constexpr int kFit = (113 * 1024 - 1024 - 256) / kStageBytes;  // two CTAs an SM
  static constexpr int kStages = kFit > 6 ? 6 : kFit < 2 ? 2 : kFit;
  static constexpr int kRing = kStages * kStageBytes;
  static constexpr int kSmemBytes = 1024 + kRing + (2 * kStages + 1) * 8 + 16;
  static constexpr int kPerSm = 228 * 1024 / (kSmemBytes + 1024) < 2 ? 1 : 2;
  static_assert(kPartBytes + mx::slot_rows(BN, kMaxSplits) * kPartCols * 4 <= kRing, "parts");
  static_assert(kSmemBytes <= kMaxDynamicSmem, "shared memory budget");
};

struct W4Args {
  Tail out;
  int stages;
  int tiles_m;
  int zeros;      // zero points are given
  int tile_cols;  // columns of the output per tile: 128, gated 64
  int stream_w;
  int* status;
  uint64_t timeout_ns;
};

struct Maps {  // of the two halves of a tile's weights
  CUtensorMap W[2], S[2], Z[2], X;
};

// D += A B, m16n8k16, fp32 sums.
template <class T>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same<T, __half>::value)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A zero point as what dequantize8 subtracts, twice in a word: of 1024 + code (fp16)
// or 128 + code (bf16), the numbers whose last mantissa bits are the code.
template <class T>
__device__ __forceinline__ uint32_t zero_pair(uint32_t z) {
  return (z | (std::is_same<T, __half>::value ? 0x6400u : 0x4300u)) * 0x10001u;
}

// The 8 codes of a word minus the zero point, in pairs of neighbours.
template <class T>
__device__ __forceinline__ void dequantize8(uint32_t w, uint32_t zero, uint32_t (&p)[4]) {
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

__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t lds_u8(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
template <class T>
__device__ __forceinline__ float lds_scale(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
  return mx::unpack2<T>(v).x;
}

template <class T, int BN, int GROUP>
__global__ void __launch_bounds__(kThreads, 2)
    ff_w4_kernel(const __grid_constant__ Maps maps, const W4Args a) {
  using C = Cfg<BN, GROUP>;
  constexpr int kStages = C::kStages;
  constexpr int kTiles = BN / 8;            // of the MMA's N
  constexpr int kGroupChunks = GROUP / 32;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* smW = smem;                             // [stage][128 rows][128 bytes], swizzled
  uint8_t* smX = smW + kStages * kWBytes;          // [stage][chunk][BN rows][32 columns]
  uint8_t* smS = smX + kStages * C::kXBytes;       // [stage][half][group][64 rows]
  uint8_t* smZ = smS + kStages * C::kSBytes;       // the same, bytes
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kRing);
  uint64_t* empty = full + kStages;
  uint64_t* received = empty + kStages;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(received + 1);

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);  // uniform
  const int lane = threadIdx.x & 31;
  const int splits = static_cast<int>(mx::cluster_size());
  const int rank = static_cast<int>(cluster_ctarank());
  const int tile = static_cast<int>(blockIdx.x) / splits;
  const int mt = tile % a.tiles_m, nt = tile / a.tiles_m;
  const int m0 = mt * BN, n0 = nt * a.tile_cols;
  const int rows = min(BN, a.out.M - m0);
  const int s_begin = static_cast<int>(static_cast<int64_t>(a.stages) * rank / splits);
  const int s_end = static_cast<int>(static_cast<int64_t>(a.stages) * (rank + 1) / splits);
  const bool pull = rows <= kPullRows;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kWarps);
    }
    mbar_init(received, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  __syncthreads();
  grid_dependency_trigger();
  grid_dependency_wait();

  if (warp == kWarps) {
    int stage = 0;
    uint32_t phase = 0, armed = 0, parity = 0;
    bool ok = true;
    const uint64_t policy = l2_policy_evict_first();
    const uint32_t bytes = C::kStageBytes - (a.zeros ? 0 : C::kZBytes);
    for (int s = s_begin; s < s_end; ++s) {
      ok = mx::mbar_wait_warp(&empty[stage], phase ^ 1u, abort_flag, a.timeout_ns);
      if (!ok) break;
      if (mx::elect_one()) {
        mbar_arrive_expect_tx(&full[stage], bytes);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          // the second half: the next 64 rows, or (gated) the same of the other weight
          const int n = n0 + (a.out.gated ? 0 : h * kHalfRows);
          uint8_t* w = smW + stage * kWBytes + h * (kWBytes / 2);
          if (a.stream_w)
            tma_load_2d_hint(&maps.W[h], &full[stage], w, s * (kStageK / 2), n, policy);
          else
            tma_load_2d(&maps.W[h], &full[stage], w, s * (kStageK / 2), n);
          tma_load_2d(&maps.S[h], &full[stage], smS + stage * C::kSBytes + h * (C::kSBytes / 2), n,
                      s * C::kGroups);
          if (a.zeros)
            tma_load_2d(&maps.Z[h], &full[stage], smZ + stage * C::kZBytes + h * (C::kZBytes / 2),
                        n, s * C::kGroups);
        }
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
          tma_load_2d(&maps.X, &full[stage], smX + stage * C::kXBytes + c * (BN * 64),
                      s * kStageK + c * 32, m0);
      }
      __syncwarp();
      armed |= 1u << stage;
      parity = (parity & ~(1u << stage)) | (phase << stage);
      if (++stage == kStages) {
        stage = 0;
        phase ^= 1u;
      }
    }
    if (!ok) {
      if (lane == 0)
        raise_abort(a.status, abort_flag, kStatusTimeoutBase | (kRoleProducer << 4) | 1);
      // let every load already issued land before shared memory is released
      for (int s = 0; s < kStages; ++s)
        if (armed & (1u << s)) (void)mbar_wait(&full[s], (parity >> s) & 1u, nullptr, a.timeout_ns);
      __syncwarp();
    }
    if (splits > 1) mx::cluster_arrive_relaxed();
  } else {
    const int g = lane >> 2, t = lane & 3;
    const int row = warp * 16 + g;  // this thread's rows of the tile: row and row + 8
    const uint32_t w_off = static_cast<uint32_t>(row * 128 + 4 * t);
    const uint32_t x_off = static_cast<uint32_t>(g * 64 + 16 * t);
    const uint32_t swizzle = static_cast<uint32_t>(g << 4);
    // scales and zero points: [half][group][64 rows]
    const uint32_t s_row = static_cast<uint32_t>((row >> 6) * C::kGroups * 64 + (row & 63));
    float acc[kTiles][4] = {};
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int s = s_begin; s < s_end; ++s) {
      ok = mx::mbar_wait_warp(&full[stage], phase, abort_flag, a.timeout_ns);
      if (!ok) break;
      const uint32_t w_at = smem_u32(smW + stage * kWBytes) + w_off;
      const uint32_t x_at = smem_u32(smX + stage * C::kXBytes) + x_off;
      const uint32_t s_at = smem_u32(smS + stage * C::kSBytes) + 2 * s_row;
      const uint32_t z_at = smem_u32(smZ + stage * C::kZBytes) + s_row;
#pragma unroll
      for (int gr = 0; gr < C::kGroups; ++gr) {
        float sum[kTiles][4] = {};
        uint32_t z0 = 8, z1 = 8;
        if (a.zeros) {
          z0 = lds_u8(z_at + gr * 64);
          z1 = lds_u8(z_at + gr * 64 + 8);
        }
        z0 = zero_pair<T>(z0);
        z1 = zero_pair<T>(z1);
#pragma unroll
        for (int j = 0; j < kGroupChunks; ++j) {
          const int c = gr * kGroupChunks + j;
          const uint32_t at = w_at + ((static_cast<uint32_t>(c) << 4) ^ swizzle);
          uint32_t p[4], q[4];
          dequantize8<T>(lds32(at), z0, p);
          dequantize8<T>(lds32(at + 1024), z1, q);
#pragma unroll
          for (int i = 0; i < kTiles; ++i) {
            const uint4 x = lds128(x_at + c * (BN * 64) + i * 512);
            mma16816<T>(sum[i], p[0], q[0], p[1], q[1], x.x, x.y);
            mma16816<T>(sum[i], p[2], q[2], p[3], q[3], x.z, x.w);
          }
        }
        const float s0 = lds_scale<T>(s_at + gr * 128), s1 = lds_scale<T>(s_at + gr * 128 + 16);
#pragma unroll
        for (int i = 0; i < kTiles; ++i) {
          acc[i][0] = fmaf(s0, sum[i][0], acc[i][0]);
          acc[i][1] = fmaf(s0, sum[i][1], acc[i][1]);
          acc[i][2] = fmaf(s1, sum[i][2], acc[i][2]);
          acc[i][3] = fmaf(s1, sum[i][3], acc[i][3]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[stage]);
      if (++stage == kStages) {
        stage = 0;
        phase ^= 1u;
      }
    }
    if (!ok && lane == 0)
      raise_abort(a.status, abort_flag, kStatusTimeoutBase | (kRoleMma << 4) | 1);
    // every stage of this CTA has landed and has been read by all of its warps: the
    // ring is free for its part, and for what others send
    named_bar_sync(1, 32 * kWarps);
    if (splits > 1 && !pull) mx::cluster_arrive();
    float* part = reinterpret_cast<float*>(smem) + row;
#pragma unroll
    for (int i = 0; i < kTiles; ++i) {
      const int m = i * 8 + 2 * t;
      if (m < rows) {
        part[m * kPartCols] = acc[i][0];
        part[m * kPartCols + 8] = acc[i][2];
      }
      if (m + 1 < rows) {
        part[(m + 1) * kPartCols] = acc[i][1];
        part[(m + 1) * kPartCols + 8] = acc[i][3];
      }
    }
    __syncwarp();
    if (splits > 1 && pull) mx::cluster_arrive();  // the part is there to be read
  }
  __syncwarp();
  join_and_finish<BN, kThreads>(a.out, smem, received, abort_flag, a.status, a.timeout_ns, rank,
                                splits, m0, n0, rows);
}

// Into how many parts of at least two stages K is divided: as many as run in one wave.
template <class T, int BN, int GROUP>
int choose_splits(int64_t tiles, int64_t stages, const DeviceCtx& d) {
  using C = Cfg<BN, GROUP>;
  static Residency residency[64];
  int splits = 1;
  for (int c = 2; c <= kMaxSplits && stages >= 2 * c; ++c) {
    const int n =
        residency[d.device & 63].of(c, ff_w4_kernel<T, BN, GROUP>, kThreads, C::kSmemBytes, d);
    if (tiles <= static_cast<int64_t>(n) * C::kPerSm) splits = c;
  }
  return splits;
}

template <class T, int BN, int GROUP>
bool set_attributes(const DeviceCtx& d) {
  static std::atomic<uint64_t> attr_done{0};
  const void* kern = reinterpret_cast<const void*>(ff_w4_kernel<T, BN, GROUP>);
  const uint64_t bit = 1ull << (d.device & 63);
  if (!(attr_done.load(std::memory_order_acquire) & bit)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Cfg<BN, GROUP>::kSmemBytes) != cudaSuccess ||
        cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared) != cudaSuccess)
      return false;
    attr_done.fetch_or(bit, std::memory_order_acq_rel);
  }
  return true;
}

template <class T, int BN, int GROUP>
int launch(const W4Problem& p, const DeviceCtx& d) {
  using C = Cfg<BN, GROUP>;
  if (!set_attributes<T, BN, GROUP>(d)) return runtime_error();
  const int64_t row_bytes = (p.K + 7) / 8 * 4, groups = (p.K + GROUP - 1) / GROUP;
  Maps maps;
  int rc = encode_tmap_rows(&maps.X, p.X, 2, p.K, p.M, p.ldx, 32, BN);
  for (int h = 0; h < 2 && rc == 0; ++h) {
    const W4Weight& w = p.w[p.gated ? h : 0];
    rc = encode_tmap_u8_2d(&maps.W[h], w.Q, row_bytes, p.N, w.ldq, kHalfRows);
    if (rc == 0)
      rc = encode_tmap_rows(&maps.S[h], w.S, 2, p.N, groups, w.lds, kHalfRows, C::kGroups);
    maps.Z[h] = maps.S[h];  // (not used without zero points)
    if (rc == 0 && w.Z != nullptr)
      rc = encode_tmap_rows(&maps.Z[h], w.Z, 1, p.N, groups, w.ldz, kHalfRows, C::kGroups);
  }
  if (rc != 0) return rc;
  const int tile_cols = p.gated ? kHalfRows : kPartCols;
  const int64_t tiles_m = (p.M + BN - 1) / BN;
  const int64_t tiles = tiles_m * ((p.N + tile_cols - 1) / tile_cols);
  const int64_t stages = (p.K + kStageK - 1) / kStageK;
  const int splits = choose_splits<T, BN, GROUP>(tiles, stages, d);
  if (tiles * splits > INT32_MAX) return GEMM_ERR_INVALID_ARG;
  W4Args a{};
  a.out = Tail{static_cast<uint16_t*>(p.Y),
               static_cast<const uint16_t*>(p.bias),
               nullptr,
               nullptr,
               p.ldy,
               0,
               0,
               static_cast<int>(p.M),
               static_cast<int>(p.N),
               p.dtype,
               p.act,
               p.gated};
  a.stages = static_cast<int>(stages);
  a.tiles_m = static_cast<int>(tiles_m);
  a.zeros = p.w[0].Z != nullptr;
  a.tile_cols = tile_cols;
  a.stream_w = tiles_m == 1;
  a.status = d.status;
  a.timeout_ns = d.timeout_ns;
  Launch l(dim3(static_cast<unsigned>(tiles * splits)), dim3(kThreads), C::kSmemBytes, p.stream);
  l.cluster(static_cast<unsigned>(splits));
  return launched(cudaLaunchKernelEx(&l.cfg, ff_w4_kernel<T, BN, GROUP>, maps, a));
}

template <class T, int GROUP>
int launch_rows(const W4Problem& p, const DeviceCtx& d) {
  if (p.M <= 8) return launch<T, 8, GROUP>(p, d);
  if (p.M <= 16) return launch<T, 16, GROUP>(p, d);
  if (p.M <= 32) return launch<T, 32, GROUP>(p, d);
  return launch<T, 64, GROUP>(p, d);
}

template <class T>
int launch_group(const W4Problem& p, const DeviceCtx& d) {
  switch (p.group) {
    case 32: return launch_rows<T, 32>(p, d);
    case 64: return launch_rows<T, 64>(p, d);
    default: return launch_rows<T, 128>(p, d);
  }
}

}  // namespace

int launch_w4(const W4Problem& p, const DeviceCtx& d) {
  return p.dtype == MX_F16 ? launch_group<__half>(p, d) : launch_group<__nv_bfloat16>(p, d);
}

}  // namespace ff
}  // namespace ttc
