// C = act(A B^T + bias) for MX operands, small and middling shapes: swap-AB
// tiles with K split over a cluster.
//
// A tile is 128 rows of B (columns of C, the MMA's M) by BN rows of A (the
// MMA's N: 16 to 64), so a single token wastes none of the weight's
// bandwidth.  The K range of a tile is split over the CTAs of a cluster; each
// accumulates its part in TMEM and puts it in its own shared memory, sends
// every other CTA the rows that one owns (one bulk copy between the SMs'
// shared memories each), and adds the parts of its own rows in rank order.
// Nothing is kept in device memory between or during calls (no workspace, no
// counters), and the order of the sums is fixed by the shape.  Up to 4 rows the
// parts are read from the other CTAs' shared memory instead of sent: loads run
// at some 8 bytes a clock and SM, too slow for more rows (60 x 4096 x 8192 MXFP8:
// 15.0 us, 11.6 with copies when this was tried), but a few rows would wait
// longer for the copies (1 x 8192 x 4096 MXFP8: 8.6 us, 9.2 with copies then;
// 8.5 now).
//
// Bound by reading B from device memory where it is large (32 x 28672 x 8192
// MXFP4: 22.8 us, 5.5 TB/s; 1 x 28672 x 4096 MXFP8: 21.6 us, 5.6 TB/s), else by a
// chain of 4 us (1 x 1024 x 1024 MXFP8) to 6 us: launch, first load, accumulator,
// joining, store.
//
//   warp 0   TMA producer: elements by tensor maps into 128-byte-swizzled
//            shared memory, scale tiles by plain bulk copies
//   warp 1   TMEM allocation; scale tiles to TMEM (tcgen05.cp) and the
//            block-scaled tcgen05.mma
//   warps 2-5  accumulator -> shared memory; then all warps: sum, bias,
//            activation, store
#include <atomic>

#include "mx_internal.h"
#include "mx_umma.cuh"

namespace ttc {
namespace mx {
namespace {

constexpr int kThreads = 192;
constexpr int kTileN = 128;  // columns of C per tile
constexpr int kMaxSplits = 8;  // CTAs of a cluster
constexpr int kPullRows = 4;  // up to so many rows the parts are read, not sent

template <int FMT, int BN, bool DEEP>
struct SplitCfg {
  // one CTA an SM with a deep ring, or two
  static constexpr int kStages = DEEP ? (BN == 16 ? 10 : BN == 32 ? 9 : 8) : (BN == 64 ? 4 : 5);
  static constexpr int kWBytes = kTileN * kRowBytes;
  static constexpr int kXBytes = BN * kRowBytes;
  static constexpr int kSfBytes = Kind<FMT>::kSfTiles * kTileBytes;
  static constexpr int kStageBytes = kWBytes + kXBytes + 2 * kSfBytes;
  // over the ring: this CTA's fp32 part of the tile, then the parts of its rows
  // that the others send
  static constexpr int kPartBytes = BN * kTileN * 4;
  static constexpr int kRing = kStages * kStageBytes;
  static constexpr int kSmemBytes = 1024 + kRing + (2 * kStages + 3) * 8 + 16;
  static_assert(kPartBytes + slot_rows(BN, kMaxSplits) * kTileN * 4 <= kRing, "parts");
  // accumulator, then one set of scales per stage: a stage's columns are
  // written again only after the MMAs that read them have completed
  static constexpr int kSfBase = BN < 32 ? 32 : BN;
  static constexpr int kCols = kSfBase + kStages * 2 * Kind<FMT>::kSfCols;
  static constexpr uint32_t kTmemCols = kCols <= 64 ? 64 : kCols <= 128 ? 128 : 256;
  // CTAs an SM holds at once (228 KiB of shared memory, 1 KiB of it per CTA
  // the system's; 512 TMEM columns)
  static constexpr int kPerSm = 228 * 1024 / (kSmemBytes + 1024) < 512 / static_cast<int>(kTmemCols)
                                    ? 228 * 1024 / (kSmemBytes + 1024)
                                    : 512 / static_cast<int>(kTmemCols);
  static_assert(kCols <= 256, "TMEM columns");
  static_assert(kSmemBytes <= kMaxDynamicSmem, "shared memory budget");
};

struct SplitArgs {
  const uint8_t *SB, *SA;
  Output out;
  int row_bytes;  // bytes of a row of elements
  int tiles;      // scale tiles along K
  int stages;     // ring stages along K
  int tiles_m;
  int stream_b;   // B is read once: let L2 drop it first
  int* status;
  uint64_t timeout_ns;
};

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

template <int FMT, int BN, bool DEEP>
__global__ void __launch_bounds__(kThreads)
    split_gemm_kernel(const __grid_constant__ CUtensorMap tmB,
                      const __grid_constant__ CUtensorMap tmA, const SplitArgs a) {
  using Cfg = SplitCfg<FMT, BN, DEEP>;
  constexpr int kStages = Cfg::kStages;
  constexpr int kSfTiles = Kind<FMT>::kSfTiles;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* smW = smem;
  uint8_t* smX = smW + kStages * Cfg::kWBytes;
  uint8_t* smS = smX + kStages * Cfg::kXBytes;  // per stage: scales of B, scales of A
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + Cfg::kRing);
  uint64_t* empty = full + kStages;
  uint64_t* acc_full = empty + kStages;
  uint64_t* drain = acc_full + 1;
  uint64_t* received = drain + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(received + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);  // uniform
  const int lane = threadIdx.x & 31;
  const int splits = static_cast<int>(cluster_size());
  const int rank = static_cast<int>(cluster_ctarank());
  const int tile = static_cast<int>(blockIdx.x) / splits;
  const int mt = tile % a.tiles_m, nt = tile / a.tiles_m;
  const int m0 = mt * BN, n0 = nt * kTileN;
  const int rows = min(BN, a.out.M - m0);
  const int s_begin = static_cast<int>(static_cast<int64_t>(a.stages) * rank / splits);
  const int s_end = static_cast<int>(static_cast<int64_t>(a.stages) * (rank + 1) / splits);

  // the rows of the tile that rank r finishes are [first_row(r), first_row(r + 1))
  auto first_row = [&](int r) { return rows * r / splits; };
  const int r0 = first_row(rank), r1 = first_row(rank + 1);
  const int slot_bytes = (BN + splits - 1) / splits * kTileN * 4;
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
    tma_prefetch_desc(&tmB);
    tma_prefetch_desc(&tmA);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, Cfg::kTmemCols);
    tmem_relinquish_alloc_permit();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  grid_dependency_trigger();
  grid_dependency_wait();
  const int c = static_cast<int>(threadIdx.x & 15) * 8;  // the columns this thread finishes
  const uint4 bias = load_bias(a.out, n0 + c);

  if (warp == 0) {
    int stage = 0;
    uint32_t phase = 0, armed = 0, parity = 0;
    bool ok = true;
    const uint64_t policy = l2_policy_evict_first();
    const uint8_t* sb = a.SB + static_cast<int64_t>(nt) * a.tiles * kTileBytes;
    const uint8_t* sa = a.SA + static_cast<int64_t>(m0 / kTileRows) * a.tiles * kTileBytes;
    for (int s = s_begin; s < s_end; ++s) {
      ok = mbar_wait_warp(&empty[stage], phase ^ 1u, abort_flag, a.timeout_ns);
      if (!ok) break;
      if (elect_one()) {
        // the last stage may have one scale tile of two
        const int kt = s * kSfTiles;
        const uint32_t sf = static_cast<uint32_t>(min(kSfTiles, a.tiles - kt)) * kTileBytes;
        mbar_arrive_expect_tx(&full[stage], Cfg::kWBytes + Cfg::kXBytes + 2 * sf);
        uint8_t* w = smW + stage * Cfg::kWBytes;
        if (a.stream_b)
          tma_load_2d_hint(&tmB, &full[stage], w, s * kRowBytes, n0, policy);
        else
          tma_load_2d(&tmB, &full[stage], w, s * kRowBytes, n0);
        tma_load_2d(&tmA, &full[stage], smX + stage * Cfg::kXBytes, s * kRowBytes, m0);
        uint8_t* sfw = smS + stage * 2 * Cfg::kSfBytes;
        bulk_load(sfw, sb + static_cast<int64_t>(kt) * kTileBytes, sf, &full[stage]);
        bulk_load(sfw + Cfg::kSfBytes, sa + static_cast<int64_t>(kt) * kTileBytes, sf,
                  &full[stage]);
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
    if (splits > 1) cluster_arrive_relaxed();
  } else if (warp == 1) {
    const uint32_t base = __shfl_sync(0xffffffffu, tmem, 0);
    // rows 64 .. 127 of a scale tile are its columns 2 and 3
    const uint32_t half = BN == 64 ? static_cast<uint32_t>(mt & 1) * 2u : 0u;
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int s = s_begin; s < s_end; ++s) {
      ok = mbar_wait_warp(&full[stage], phase, abort_flag, a.timeout_ns);
      if (!ok) break;
      tc_fence_after_sync();
      if (elect_one()) {
        const uint32_t s_addr = smem_u32(smS + stage * 2 * Cfg::kSfBytes);
        const uint32_t sfw = base + Cfg::kSfBase + stage * 2 * Kind<FMT>::kSfCols;
        const uint32_t sfx = sfw + Kind<FMT>::kSfCols;
        // (a second tile that the last k-block does not have is copied and not used)
#pragma unroll
        for (int t = 0; t < kSfTiles; ++t) {
          copy_scales<1>(sfw + 4 * t, (s_addr + t * kTileBytes) >> 4);
          copy_scales<1>(sfx + 4 * t, (s_addr + Cfg::kSfBytes + t * kTileBytes) >> 4);
        }
        issue_mmas<FMT, 1, kTileN, BN, 4>(base, smem_u32(smW + stage * Cfg::kWBytes),
                                          smem_u32(smX + stage * Cfg::kXBytes), sfw, sfx + half,
                                          a.row_bytes - s * kRowBytes, s != s_begin);
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
    if (splits > 1) cluster_arrive_relaxed();
  } else {
    int ok = 1;
    if (lane == 0) ok = mbar_wait(acc_full, 0, abort_flag, a.timeout_ns) ? 1 : 0;
    ok = __shfl_sync(0xffffffffu, ok, 0);
    // all loads have landed and all MMAs have read them: the ring is free, for
    // what others send, too
    if (splits > 1 && !pull) cluster_arrive_relaxed();
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
          if (r + i < rows) part[(r + i) * kTileN] = __uint_as_float(v[i]);
      }
    } else if (lane == 0) {
      raise_abort(a.status, abort_flag, kStatusTimeoutBase | (kRoleEpilogue << 4) | 1);
    }
    __syncwarp();
    if (splits > 1 && pull) cluster_arrive();  // the part is there to be read
  }
  __syncwarp();
  tc_fence_before_sync();
  uint8_t* incoming = smem + Cfg::kPartBytes;
  if (splits > 1) {
    fence_proxy_async_smem();  // the part is read by bulk copies
    __syncthreads();           // all of this CTA's part is written
    cluster_wait();            // pull: all parts are; push: all rings are free
    if (!pull && threadIdx.x == 0) {
      mbar_arrive_expect_tx(received,
                            static_cast<uint32_t>((splits - 1) * (r1 - r0) * kTileN * 4));
      for (int k = 1; k < splits && *abort_flag == 0; ++k) {
        const int to = rank + k < splits ? rank + k : rank + k - splits;
        const int from_row = first_row(to), n = first_row(to + 1) - from_row;
        if (n == 0) continue;
        // the receiver keeps its slots in rank order, without its own
        const int slot = rank < to ? rank : rank - 1;
        bulk_push(map_to_cta(smem_u32(incoming) + static_cast<uint32_t>(slot * slot_bytes),
                             static_cast<uint32_t>(to)),
                  smem + from_row * kTileN * 4, static_cast<uint32_t>(n * kTileN * 4),
                  map_to_cta(smem_u32(received), static_cast<uint32_t>(to)));
      }
    }
    // (after an abort, too: what others have sent has to land before this CTA ends)
    if (!pull && r1 > r0 && !mbar_wait(received, 0, nullptr, a.timeout_ns))
      raise_abort(a.status, abort_flag, kStatusTimeoutBase | (kRoleEpilogue << 4) | 2);
  } else {
    __syncthreads();
  }

  const bool aborted = *abort_flag != 0;
  if (splits > 1 && pull) {
    // items: 8 columns of a row, at most one for a thread of the cluster
    static_assert(kPullRows * (kTileN / 8) <= kThreads, "an item a thread");
    const int m = threadIdx.x >> 4;
    const bool mine = rank == 0 && m < rows && n0 + c < a.out.N;
    float v[8] = {};
    if (mine) {
      float4 p[kMaxSplits][2];  // all parts are on their way before the first is added
#pragma unroll
      for (int s = 0; s < kMaxSplits; ++s) {
        if (s >= splits) break;
        const uint32_t src = map_to_cta(
            smem_u32(smem) + static_cast<uint32_t>(m * kTileN + c) * 4, static_cast<uint32_t>(s));
        p[s][0] = ld_cluster_f4(src);
        p[s][1] = ld_cluster_f4(src + 16);
      }
#pragma unroll
      for (int s = 0; s < kMaxSplits; ++s) {
        if (s >= splits) break;
        add8(v, p[s][0], p[s][1]);
      }
    }
    __syncwarp();
    // The others' parts have been read: a release, since the loads above have to
    // be over before their owners leave.  Only this CTA has read any.  (1 x 1024 x
    // 1024 MXFP8: 3.97 us, 4.10 where all release, 3.84 without an order; 2 x 2048 x
    // 8192: 6.66, 6.91 and 6.65.)
    if (rank == 0)
      cluster_arrive();
    else
      cluster_arrive_relaxed();
    if (mine && !aborted)
      with_columns(a.out, n0 + c, bias, [&](const auto& columns, auto act) {
        columns.template store<decltype(act)::value>(m0 + m, v);
      });
  } else {
    __syncwarp();
    if (splits > 1) cluster_arrive_relaxed();  // what was sent here has left the others' memory
    if (!aborted)
      finish_rows<kThreads>(a.out, m0 + r0, n0 + c, r1 - r0, bias, splits, [&](int s) {
        return reinterpret_cast<const float*>(
                   s == rank ? smem + r0 * kTileN * 4
                             : incoming + (s < rank ? s : s - 1) * slot_bytes) + c;
      });
  }
  __syncwarp();
  // no CTA leaves while another, or its own copies, may still read its shared memory
  if (splits > 1)
    cluster_wait();
  else
    __syncthreads();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, Cfg::kTmemCols);
  }
}

// Into how many parts of at least four k-blocks K is divided: as many as run in
// one wave, since a second wave costs more than the division brings (32 x 8192
// x 4096 MXFP8, 64 tiles: 1 part 11.7 us, 2 parts 10.5, 4 parts 10.0, 5 parts 15.1).
template <int FMT, int BN, bool DEEP>
int choose_splits(int64_t tiles, int64_t stages, const DeviceCtx& d) {
  using Cfg = SplitCfg<FMT, BN, DEEP>;
  static Residency residency[64];
  int splits = 1;
  for (int c = 2; c <= kMaxSplits && stages >= 4 * c; ++c) {
    const int n = residency[d.device & 63].of(c, split_gemm_kernel<FMT, BN, DEEP>, kThreads,
                                              Cfg::kSmemBytes, d);
    if (tiles <= static_cast<int64_t>(n) * Cfg::kPerSm) splits = c;
  }
  return splits;
}

template <int FMT, int BN, bool DEEP>
bool set_attributes(const DeviceCtx& d) {
  static std::atomic<uint64_t> attr_done{0};
  auto kern = split_gemm_kernel<FMT, BN, DEEP>;
  using Cfg = SplitCfg<FMT, BN, DEEP>;
  const uint64_t bit = 1ull << (d.device & 63);
  if (!(attr_done.load(std::memory_order_acquire) & bit)) {
    if (cudaFuncSetAttribute(reinterpret_cast<const void*>(kern),
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Cfg::kSmemBytes) != cudaSuccess ||
        // several CTAs an SM: all of the SM's memory as shared memory
        cudaFuncSetAttribute(reinterpret_cast<const void*>(kern),
                             cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared) != cudaSuccess)
      return false;
    attr_done.fetch_or(bit, std::memory_order_acq_rel);
  }
  return true;
}

template <int FMT, int BN, bool DEEP>
int launch(const MxGemmProblem& p, const DeviceCtx& d, int splits) {
  using Cfg = SplitCfg<FMT, BN, DEEP>;
  auto kern = split_gemm_kernel<FMT, BN, DEEP>;
  const int64_t row_bytes = mx_row_bytes(p.K, FMT);
  CUtensorMap tB, tA;
  int rc = encode_tmap_u8_2d(&tB, p.B, row_bytes, p.N, p.ldb, kTileN);
  if (rc == 0) rc = encode_tmap_u8_2d(&tA, p.A, row_bytes, p.M, p.lda, BN);
  if (rc != 0) return rc;
  const int64_t stages = (row_bytes + kRowBytes - 1) / kRowBytes;
  const int64_t tiles_m = (p.M + BN - 1) / BN;
  const int64_t tiles = tiles_m * ((p.N + kTileN - 1) / kTileN);
  if (tiles * splits > INT32_MAX) return GEMM_ERR_INVALID_ARG;
  const SplitArgs a{static_cast<const uint8_t*>(p.SB),
                    static_cast<const uint8_t*>(p.SA),
                    output_of(p),
                    static_cast<int>(row_bytes),
                    static_cast<int>(scale_tiles(p.K)),
                    static_cast<int>(stages),
                    static_cast<int>(tiles_m),
                    tiles_m == 1,
                    d.status,
                    d.timeout_ns};
  Launch l(dim3(static_cast<unsigned>(tiles * splits)), dim3(kThreads), Cfg::kSmemBytes, p.stream);
  l.cluster(static_cast<unsigned>(splits));
  const cudaError_t e = cudaLaunchKernelEx(&l.cfg, kern, tB, tA, a);
  return launched(e);
}

template <int FMT, int BN, bool DEEP>
int launch_depth(const MxGemmProblem& p, const DeviceCtx& d, int64_t tiles) {
  if (!set_attributes<FMT, BN, DEEP>(d)) return runtime_error();
  const int64_t stages = (mx_row_bytes(p.K, FMT) + kRowBytes - 1) / kRowBytes;
  return launch<FMT, BN, DEEP>(p, d, choose_splits<FMT, BN, DEEP>(tiles, stages, d));
}

// Where the tiles alone give most SMs one CTA, one with a deep ring and the
// whole of K; else two an SM, which also cover each other's ends (32 x 14336 x
// 4096 MXFP8, 112 tiles: 12.7 us, 14.0 with two; 32 x 28672 x 8192 MXFP4, 224
// tiles: 26.6 us, 22.2 with two).
template <int FMT, int BN>
int launch_tile(const MxGemmProblem& p, const DeviceCtx& d) {
  const int64_t tiles = (p.M + BN - 1) / BN * ((p.N + kTileN - 1) / kTileN);
  return tiles > d.sm_count / 2 && tiles <= d.sm_count ? launch_depth<FMT, BN, true>(p, d, tiles)
                                                       : launch_depth<FMT, BN, false>(p, d, tiles);
}

template <int FMT>
int launch_rows(const MxGemmProblem& p, const DeviceCtx& d) {
  if (p.M <= 16) return launch_tile<FMT, 16>(p, d);
  if (p.M <= 32) return launch_tile<FMT, 32>(p, d);
  return launch_tile<FMT, 64>(p, d);
}

template <class T>
__global__ void bias_fill_kernel(uint16_t* C, const uint16_t* bias, int64_t M, int64_t N,
                                 int64_t ldc, int act) {
  const int64_t total = M * N;
  grid_dependency_trigger();
  grid_dependency_wait();
  for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t r = i / N, c = i - r * N;
    const float b = bias != nullptr ? unpack2<T>(bias[c]).x : 0.0f;
    const float2 y = finish2(make_float2(b, b), make_float2(0.0f, 0.0f), act);
    C[r * ldc + c] = static_cast<uint16_t>(pack2<T>(y.x, y.x));
  }
}

}  // namespace

int launch_mx_split_gemm(const MxGemmProblem& p, const DeviceCtx& d) {
  return p.format == MX_FP8 ? launch_rows<MX_FP8>(p, d) : launch_rows<MX_FP4>(p, d);
}

int launch_mx_bias_fill(const MxGemmProblem& p) {
  const int64_t blocks = (p.M * p.N + 255) / 256;
  Launch l(dim3(static_cast<unsigned>(blocks < 4096 ? blocks : 4096)), dim3(256), 0, p.stream);
  uint16_t* c = static_cast<uint16_t*>(p.C);
  const uint16_t* b = static_cast<const uint16_t*>(p.bias);
  const cudaError_t e = p.dtype == MX_F16 ? cudaLaunchKernelEx(&l.cfg, bias_fill_kernel<__half>, c,
                                                               b, p.M, p.N, p.ldc, p.act)
                                          : cudaLaunchKernelEx(&l.cfg,
                                                               bias_fill_kernel<__nv_bfloat16>, c,
                                                               b, p.M, p.N, p.ldc, p.act);
  return launched(e);
}

}  // namespace mx
}  // namespace ttc
