// 16-bit products of few rows: swap-AB tiles with K split over a cluster, for the
// gated projections and for dX = dG Wg + dU Wu (ff_internal.h, kGated and kConcat).
//
// A tile is 128 rows of the weights (the MMA's M) by BN rows of x (its N, 16 to
// 128), so that few rows waste none of the weights' bandwidth.  The gated form's 128
// are 64 of the gate and the same 64 of the other projection: both lie in one
// accumulator, and the sums meet in the epilogue.  The concat form takes the
// weights MN-major as they are stored (F x D), the k-blocks of the second pair of
// operands after those of the first.  The K range of a tile is divided among the
// CTAs of a cluster, whose parts are joined in shared memory (ff_common.cuh):
// nothing is kept in device memory, and the order of the sums is fixed by the shape and the
// number of parts, which is the same for every call of a shape on one GPU.
//
//   warp 0     TMA producer into a ring of 128-byte-swizzled stages
//   warp 1     TMEM, tcgen05.mma
//   warps 2-5  accumulator -> shared memory; then all warps finish the rows
#include <atomic>

#include "ff_common.cuh"

namespace ttc {
namespace ff {
namespace {

using mx::elect_one;
using mx::mbar_wait_warp;

constexpr int kThreads = 192;
constexpr int kBK = 64;
constexpr int kWBytes = kPartCols * kBK * 2;  // weights of a stage
constexpr int kSlab = kWBytes / 2;            // 64 rows of them

template <int BN, bool DEEP>
struct Cfg {
  // one CTA an SM with a deep ring, or two
  static constexpr int kStages = DEEP ? (BN == 16 ? 12 : BN == 32 ? 11 : BN == 64 ? 9 : 7)
                                      : (BN == 16 ? 6 : BN == 32 ? 5 : 4);
  static constexpr int kXBytes = BN * kBK * 2;
  static constexpr int kStageBytes = kWBytes + kXBytes;
  static constexpr int kRing = kStages * kStageBytes;
  static constexpr int kPartBytes = BN * kPartCols * 4;
  static constexpr int kSmemBytes = 1024 + kRing + (2 * kStages + 3) * 8 + 16;
  static constexpr uint32_t kTmemCols = BN < 32 ? 32 : BN;
  static_assert(kPartBytes + mx::slot_rows(BN, kMaxSplits) * kPartCols * 4 <= kRing, "parts");
  static_assert(kSmemBytes <= kMaxDynamicSmem, "shared memory budget");
};

struct SplitArgs {
  Tail out;
  int blocks;     // k-blocks of the first operands
  int stages;     // k-blocks in all
  int tiles_m;
  int w_mn;       // weights stored K x N
  int tile_cols;  // columns of the output per tile: 128, gated 64
  int stream_w;   // the weights are read once: let L2 drop them first
  uint32_t idesc;
  int* status;
  uint64_t timeout_ns;
};

__device__ __forceinline__ void single_mma(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tmov.b64 da, {%1, %5};\n\t"
      "mov.b64 db, {%2, %5};\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "r"(mx::kDescHigh)
      : "memory");
}

template <int BN, bool DEEP>
__global__ void __launch_bounds__(kThreads)
    ff_split_kernel(const __grid_constant__ CUtensorMap tmW0,
                    const __grid_constant__ CUtensorMap tmW1,
                    const __grid_constant__ CUtensorMap tmX0,
                    const __grid_constant__ CUtensorMap tmX1, const SplitArgs a) {
  using C = Cfg<BN, DEEP>;
  constexpr int kStages = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* smW = smem;
  uint8_t* smX = smW + kStages * kWBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kRing);
  uint64_t* empty = full + kStages;
  uint64_t* acc_full = empty + kStages;
  uint64_t* drain = acc_full + 1;
  uint64_t* received = drain + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(received + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

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
      mbar_init(&empty[s], 1);
    }
    mbar_init(acc_full, 1);
    mbar_init(drain, 1);
    mbar_init(received, 1);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmW0);
    tma_prefetch_desc(&tmW1);
    tma_prefetch_desc(&tmX0);
    tma_prefetch_desc(&tmX1);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::kTmemCols);
    tmem_relinquish_alloc_permit();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  grid_dependency_trigger();
  grid_dependency_wait();

  if (warp == 0) {
    int stage = 0;
    uint32_t phase = 0, armed = 0, parity = 0;
    bool ok = true;
    const uint64_t policy = l2_policy_evict_first();
    for (int s = s_begin; s < s_end; ++s) {
      ok = mbar_wait_warp(&empty[stage], phase ^ 1u, abort_flag, a.timeout_ns);
      if (!ok) break;
      if (elect_one()) {
        mbar_arrive_expect_tx(&full[stage], C::kStageBytes);
        uint8_t* w = smW + stage * kWBytes;
        const bool second = s >= a.blocks;
        const int k = (second ? s - a.blocks : s) * kBK;
        auto load_w = [&](const CUtensorMap* map, uint8_t* to, int c0, int c1) {
          if (a.stream_w)
            tma_load_2d_hint(map, &full[stage], to, c0, c1, policy);
          else
            tma_load_2d(map, &full[stage], to, c0, c1);
        };
        if (a.w_mn) {
          load_w(second ? &tmW1 : &tmW0, w, n0, k);
          load_w(second ? &tmW1 : &tmW0, w + kSlab, n0 + 64, k);
        } else {
          load_w(&tmW0, w, k, n0);
          load_w(&tmW1, w + kSlab, k, n0);
        }
        tma_load_2d(second ? &tmX1 : &tmX0, &full[stage], smX + stage * C::kXBytes, k, m0);
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
  } else if (warp == 1) {
    const uint32_t base = __shfl_sync(0xffffffffu, tmem, 0);
    const uint32_t w_lead = a.w_mn ? (kSlab >> 4) << 16 : 1u << 16;
    const uint32_t w_step = a.w_mn ? (16 * 128) >> 4 : (16 * 2) >> 4;
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int s = s_begin; s < s_end; ++s) {
      ok = mbar_wait_warp(&full[stage], phase, abort_flag, a.timeout_ns);
      if (!ok) break;
      tc_fence_after_sync();
      if (elect_one()) {
        // (14 bits: above them the address names the CTA of the cluster, and the
        // descriptor the leading dimension)
        const uint32_t wl = ((smem_u32(smW + stage * kWBytes) >> 4) & 0x3FFFu) | w_lead;
        const uint32_t xl = mx::desc_low(smem_u32(smX + stage * C::kXBytes));
#pragma unroll
        for (int k = 0; k < kBK / 16; ++k)
          single_mma(base, wl + k * w_step, xl + k * 2, a.idesc,
                     (s != s_begin || k != 0) ? 1u : 0u);
        umma_commit(&empty[stage]);
        if (s == s_end - 1) umma_commit(acc_full);
      }
      __syncwarp();
      if (++stage == kStages) {
        stage = 0;
        phase ^= 1u;
      }
    }
    if (!ok) {
      if (elect_one()) {
        raise_abort(a.status, abort_flag, kStatusTimeoutBase | (kRoleMma << 4) | 1);
        umma_commit(drain);
        (void)mbar_wait(drain, 0, nullptr, a.timeout_ns);
      }
      __syncwarp();
    }
    if (splits > 1) mx::cluster_arrive_relaxed();
  } else {
    int ok = 1;
    if (lane == 0) ok = mbar_wait(acc_full, 0, abort_flag, a.timeout_ns) ? 1 : 0;
    ok = __shfl_sync(0xffffffffu, ok, 0);
    // all loads have landed and all MMAs have read them: the ring is free, for
    // what others send, too
    if (splits > 1 && !pull) mx::cluster_arrive_relaxed();
    if (ok) {
      tc_fence_after_sync();
      const int q = warp & 3;
      float* part = reinterpret_cast<float*>(smem) + q * 32 + lane;
      const uint32_t t_row = tmem + (static_cast<uint32_t>(q * 32) << 16);
#pragma unroll 1
      for (int r = 0; r < BN; r += 32) {
        if (r >= rows) break;
        uint32_t v[32];
        tmem_load_32x32b_x32(t_row + r, v);
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (r + i < rows) part[(r + i) * kPartCols] = __uint_as_float(v[i]);
      }
    } else if (lane == 0) {
      raise_abort(a.status, abort_flag, kStatusTimeoutBase | (kRoleEpilogue << 4) | 1);
    }
    __syncwarp();
    if (splits > 1 && pull) mx::cluster_arrive();  // the part is there to be read
  }
  __syncwarp();
  tc_fence_before_sync();
  join_and_finish<BN, kThreads>(a.out, smem, received, abort_flag, a.status, a.timeout_ns, rank,
                                splits, m0, n0, rows);
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// Into how many parts of at least four k-blocks K is divided: as many as run in one wave
// with a CTA an SM.  (Counting two an SM: 16 and 64 x 4096 -> 14336, gated, 39.9 and 41.2 us
// instead of 37.9 and 39.4; dX of 64 x 4096 <- 4096 2 us faster, of 8192 <- 8192 the same.)
template <int BN, bool DEEP>
int choose_splits(int64_t tiles, int64_t stages, const DeviceCtx& d) {
  static Residency residency[64];
  int splits = 1;
  for (int c = 2; c <= kMaxSplits && stages >= 4 * c; ++c) {
    const int n =
        residency[d.device & 63].of(c, ff_split_kernel<BN, DEEP>, kThreads,
                                    Cfg<BN, DEEP>::kSmemBytes, d);
    if (tiles <= n) splits = c;
  }
  return splits;
}

template <int BN, bool DEEP>
bool set_attributes(const DeviceCtx& d) {
  static std::atomic<uint64_t> attr_done{0};
  const void* kern = reinterpret_cast<const void*>(ff_split_kernel<BN, DEEP>);
  const uint64_t bit = 1ull << (d.device & 63);
  if (!(attr_done.load(std::memory_order_acquire) & bit)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Cfg<BN, DEEP>::kSmemBytes) != cudaSuccess ||
        // several CTAs an SM: all of the SM's memory as shared memory
        cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared) != cudaSuccess)
      return false;
    attr_done.fetch_or(bit, std::memory_order_acq_rel);
  }
  return true;
}

template <int BN, bool DEEP>
int launch(const Product& p, const DeviceCtx& d) {
  using C = Cfg<BN, DEEP>;
  if (!set_attributes<BN, DEEP>(d)) return runtime_error();
  const bool gated = p.form == kGated;
  CUtensorMap tW[2], tX[2];
  for (int i = 0; i < 2; ++i) {
    int rc = gated ? encode_tmap_f16_2d(&tW[i], p.B[i].p, p.K, p.N, p.B[i].ld, kBK, 64)
                   : encode_tmap_f16_2d(&tW[i], p.B[i].p, p.N, p.K, p.B[i].ld, 64, kBK);
    if (rc == 0) rc = encode_tmap_f16_2d(&tX[i], p.A[i].p, p.K, p.M, p.A[i].ld, kBK, BN);
    if (rc != 0) return rc;
  }
  const int tile_cols = gated ? 64 : kPartCols;
  const int64_t tiles_m = (p.M + BN - 1) / BN;
  const int64_t tiles = tiles_m * ((p.N + tile_cols - 1) / tile_cols);
  const int64_t blocks = (p.K + kBK - 1) / kBK;
  const int64_t stages = gated ? blocks : 2 * blocks;
  const int splits = choose_splits<BN, DEEP>(tiles, stages, d);
  if (tiles * splits > INT32_MAX) return GEMM_ERR_INVALID_ARG;
  SplitArgs a{};
  a.out = Tail{static_cast<uint16_t*>(const_cast<void*>(p.C[0].p)),
               nullptr,
               p.gate,
               p.up,
               p.C[0].ld,
               p.ld_gate,
               p.ld_up,
               static_cast<int>(p.M),
               static_cast<int>(p.N),
               p.dtype,
               gated ? p.act : static_cast<int>(kActNone),
               gated};
  a.blocks = static_cast<int>(blocks);
  a.stages = static_cast<int>(stages);
  a.tiles_m = static_cast<int>(tiles_m);
  a.w_mn = !gated;
  a.tile_cols = tile_cols;
  a.stream_w = tiles_m == 1;
  a.idesc = idesc_f16_f32(128, BN, !gated, false) |
            (p.dtype == MX_BF16 ? (1u << 7) | (1u << 10) : 0u);
  a.status = d.status;
  a.timeout_ns = d.timeout_ns;
  Launch l(dim3(static_cast<unsigned>(tiles * splits)), dim3(kThreads), C::kSmemBytes, p.stream);
  l.cluster(static_cast<unsigned>(splits));
  return launched(
      cudaLaunchKernelEx(&l.cfg, ff_split_kernel<BN, DEEP>, tW[0], tW[1], tX[0], tX[1], a));
}

// Where the tiles alone give most SMs one CTA, one with a deep ring and the whole of
// K; else two an SM, which also cover each other's ends.  Measured, one with a deep ring and
// two, gated, D = 4096, 1 and 64 rows: F = 6000 (94 tiles) 19.5 and 22.4 us, 20.5 and 26.3;
// 8000 (125) 24.6 and 24.7, 25.2 and 28.2; 14336 (224) 44.2 and 48.9, 39.6 and 40.7.  With K in
// parts the deep ring is ahead, too, by less (2000, 32 tiles: 9.4 and 10.7, 9.7 and 12.1; 4000,
// 63: 13.9 and 14.9, 13.9 and 16.9): not taken.
template <int BN>
int launch_tile(const Product& p, const DeviceCtx& d) {
  const int cols = p.form == kGated ? 64 : kPartCols;
  const int64_t tiles = (p.M + BN - 1) / BN * ((p.N + cols - 1) / cols);
  return tiles > d.sm_count / 2 && tiles <= d.sm_count ? launch<BN, true>(p, d)
                                                       : launch<BN, false>(p, d);
}

}  // namespace

// Tiles of 128 rows from 65 on (an SM holds one such CTA: a stage takes 32 KB).  Against 64
// rows: gated, D = 4096 -> F = 4096, 96 rows 16.5 us and 21.5, 256 rows 25.0 and 26.6; dX of 96 x
// 4096 <- 14336 42.7 and 73.8; of 96 x 1024 <- 1000 8.3 and 8.1.
int launch_split_product(const Product& p, const DeviceCtx& d) {
  if (p.M <= 16) return launch_tile<16>(p, d);
  if (p.M <= 32) return launch_tile<32>(p, d);
  if (p.M <= 64) return launch_tile<64>(p, d);
  return launch<128, true>(p, d);
}

}  // namespace ff
}  // namespace ttc
