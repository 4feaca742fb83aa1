// C = act(A B^T + bias) for MX operands, large shapes: a CTA pair per 256 x 256
// tile of C, persistent, the block-scaled tcgen05.mma.cta_group::2.
//
// The arrangement is that of the fp16 pair kernel in gemm_tile.cu (TMA
// producer, one MMA thread for both SMs, epilogue warps, grouped raster, every
// other wave sweeping K downwards); what differs is what the scales need:
//
//   * Each CTA stages 128 bytes of 128 rows of A and of 128 rows of B per
//     k-block, the scale tiles of its own rows of A, and those of all 256
//     rows of B (each SM scales its half of the rows of D by all columns).
//   * Per k-block the MMA thread copies the scale tiles of both SMs from
//     shared memory to TMEM (tcgen05.cp), then issues 4 MMAs.  Each ring stage
//     has its own scale columns, so that a stage that may be filled again
//     (its MMAs have completed) frees its columns too, and no other wait is
//     needed.
//   * TMEM holds 512 columns: two accumulators of 256 and the scales do not
//     fit, so the accumulators share kOverlap columns: buffer 0 is columns
//     0..255, buffer 1 ends where the scales begin.  Every epilogue warp takes
//     all its 64 columns into registers at once and then hands them back, so
//     the next tile's MMAs wait for the reads of a tile, not for its epilogue.
//   * 16 epilogue warps, 64 columns each: the GELU epilogue is about 21
//     instructions and two special-function results an element, nearly as long
//     as the MMAs of a 4-bit tile with K = 4096.
//
// Measured: 8192^3 MXFP8 + ReLU 362 us (3.04 PFLOP/s; 431 us back to back under
// the power cap), 8192 x 14336 x 4096 MXFP4 + bias + GELU 187 us (5.15 PFLOP/s),
// without an epilogue to speak of and K = 16384 590 us (6.52 PFLOP/s).  Bound by
// the tensor pipe at the clock that the power limit leaves (1.31 to 1.45 GHz in
// these launches): a tile of 64 k-blocks takes 34,000 cycles, its MMAs alone some
// 32,800, the hand-over of the shared columns the rest; of 16 k-blocks (K = 4096 in
// 4 bits) 9,700 for 8,200, and 10,500 with GELU, whose instructions slow the MMA
// warp's.  Asking for the next stage's barrier before this one's MMAs, and copying
// a tile's first scales before the columns are free, takes 200 cycles off a tile
// and nothing off the time.
#include "mx_internal.h"
#include "mx_umma.cuh"
#include "tile_common.cuh"

namespace ttc {
namespace mx {
namespace {

constexpr int kTile = 256;      // rows and columns of a pair's tile
constexpr int kHalf = 128;      // rows of A and of B per CTA
constexpr int kStages = 6;
constexpr int kEpiWarps = 16;   // four per TMEM lane quarter, 64 columns each
constexpr int kWarpCols = 64;
constexpr int kWarpRows = 32;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kPanelRows = 4096;  // rows of A per raster panel

template <int FMT>
struct PairCfg {
  static constexpr int kOperand = kHalf * kRowBytes;  // bytes of A, and of B, per stage
  static constexpr int kSf = Kind<FMT>::kSfTiles * kTileBytes;  // scales of 128 rows
  static constexpr int kStageBytes = 2 * kOperand + 3 * kSf;
  static constexpr int kBars = 2 * kStages + 6;
  static constexpr int kSmemBytes = 1024 + kStages * kStageBytes + kBars * 8 + 16;
  static constexpr int kSetCols = 3 * Kind<FMT>::kSfCols;  // scale columns of a k-block
  static constexpr int kSfBase = 512 - kStages * kSetCols;
  static constexpr int kAcc1 = kSfBase - kTile;  // first column of buffer 1
  static constexpr int kOverlap = kTile - kAcc1;
  // warps (of one CTA) that read a column both buffers share
  static constexpr int kSharers = 4 * ((kOverlap + kWarpCols - 1) / kWarpCols);
  static_assert(kAcc1 > 0, "TMEM columns");
  static_assert(kSmemBytes <= kMaxDynamicSmem, "shared memory budget");
};

struct PairArgs {
  uint16_t* C;
  const uint16_t* bias;
  int64_t ldc;
  int M, N;
  int row_bytes, sf_tiles, num_kb;
  int group_m;
  int wide;  // rows of C start on 32 bytes
  int* status;
  uint64_t timeout_ns;
};

// 32 aligned bytes, written once and not read again here.
__device__ __forceinline__ void store_32(void* p, const uint32_t (&h)[8], uint64_t policy) {
  asm volatile(
      "st.global.L2::cache_hint.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8}, %9;" ::"l"(p),
      "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3]), "r"(h[4]), "r"(h[5]), "r"(h[6]), "r"(h[7]),
      "l"(policy)
      : "memory");
}

// The kWarpCols fp32 accumulators of this thread's row of C: bias, activation,
// one rounding, stored 16 columns (a 32-byte sector) at a time straight from
// registers.  Staging the tile in shared memory for TMA stores takes 32 KiB
// from the operand ring and adds to the shared-memory traffic of the MMAs'
// operands.
template <class T, int ACT>
__device__ __forceinline__ void store_columns(const uint32_t (&v)[kWarpCols], const PairArgs& a,
                                              int row, int col0, uint64_t policy) {
  uint16_t* c = a.C + static_cast<int64_t>(row) * a.ldc + col0;
#pragma unroll
  for (int i = 0; i < kWarpCols; i += 16) {
    const int n = a.N - (col0 + i);
    if (n <= 0) break;
    uint4 b[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    if (a.bias != nullptr) {
      b[0] = load8(a.bias + col0 + i, n);
      if (n > 8) b[1] = load8(a.bias + col0 + i + 8, n - 8);
    }
    const uint32_t* bw = reinterpret_cast<const uint32_t*>(b);
    uint32_t h[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float2 x = make_float2(__uint_as_float(v[i + 2 * k]), __uint_as_float(v[i + 2 * k + 1]));
      if (a.bias != nullptr) x = __fadd2_rn(x, unpack2<T>(bw[k]));
      x = mx_activate2<ACT>(x);
      h[k] = pack2<T>(x.x, x.y);
    }
    if (row >= a.M) continue;
    if (n >= 16 && a.wide) {
      store_32(c + i, h, policy);
    } else {
      store8(c + i, make_uint4(h[0], h[1], h[2], h[3]), n);
      if (n > 8) store8(c + i + 8, make_uint4(h[4], h[5], h[6], h[7]), n - 8);
    }
  }
}

template <int FMT, class T, int ACT>
__global__ void __launch_bounds__(kThreads, 1)
    pair_gemm_kernel(const __grid_constant__ CUtensorMap tmA,
                     const __grid_constant__ CUtensorMap tmB,
                     const __grid_constant__ CUtensorMap tmSA,
                     const __grid_constant__ CUtensorMap tmSB, const PairArgs a) {
  using Cfg = PairCfg<FMT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* smA = smem;
  uint8_t* smB = smA + kStages * Cfg::kOperand;
  uint8_t* smS = smB + kStages * Cfg::kOperand;  // per stage: scales of A, of B's two halves
  uint64_t* full = reinterpret_cast<uint64_t*>(smS + kStages * 3 * Cfg::kSf);
  uint64_t* empty = full + kStages;
  uint64_t* acc_full = empty + kStages;   // [2]
  uint64_t* acc_empty = acc_full + 2;     // [2] a buffer has been read
  uint64_t* shared_empty = acc_empty + 2; // the columns both buffers share have been read
  uint64_t* drain = shared_empty + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(full + Cfg::kBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);  // uniform
  const int lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const bool leader = rank == 0;
  const int pair = static_cast<int>(cluster_id_x());
  const int npairs = static_cast<int>(num_clusters_x());
  const int num_m = (a.M + kTile - 1) / kTile;
  const int num_n = (a.N + kTile - 1) / kTile;
  const int num_tiles = num_m * num_n;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 2 * kEpiWarps);
    }
    mbar_init(shared_empty, 2 * Cfg::kSharers);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    tma_prefetch_desc(&tmSA);
    tma_prefetch_desc(&tmSB);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_alloc_permit_pair();
  }
  tc_fence_before_sync();
  cluster_sync();  // barriers of both CTAs initialised, TMEM of both SMs allocated
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  grid_dependency_trigger();
  grid_dependency_wait();
  const uint32_t full_leader = map_to_cta(smem_u32(full), 0);
  const uint32_t acc_empty_leader = map_to_cta(smem_u32(acc_empty), 0);
  const uint32_t shared_empty_leader = map_to_cta(smem_u32(shared_empty), 0);

  if (warp == 0) {
    // --------------------------------------------- TMA producer (both CTAs) ---
    int stage = 0;
    uint32_t phase = 0, armed = 0, parity = 0, down = 0;
    bool ok = true;
    for (int tile = pair; tile < num_tiles && ok; tile += npairs, down ^= 1u) {
      int mb, nb;
      tile_coords(tile, num_m, num_n, a.group_m, mb, nb);
      const int a_row = mb * kTile + rank * kHalf;
      const int b_row = nb * kTile + rank * kHalf;
      for (int i = 0; i < a.num_kb; ++i) {
        const int kb = down ? a.num_kb - 1 - i : i;
        ok = mbar_wait_warp(&empty[stage], phase ^ 1u, abort_flag, a.timeout_ns);
        if (!ok) break;
        if (elect_one()) {
          if (leader) mbar_arrive_expect_tx(&full[stage], 2 * Cfg::kStageBytes);
          const uint32_t bar = full_leader + stage * 8;
          const int kt = kb * Kind<FMT>::kSfTiles;
          uint8_t* sf = smS + stage * 3 * Cfg::kSf;
          tma_load_2d_pair(&tmA, bar, smA + stage * Cfg::kOperand, kb * kRowBytes, a_row);
          tma_load_2d_pair(&tmB, bar, smB + stage * Cfg::kOperand, kb * kRowBytes, b_row);
          // past the last row of tiles these read another row's or zeros: the
          // rows and columns they scale are not stored
          tma_load_2d_pair(&tmSA, bar, sf, 0, (2 * mb + rank) * a.sf_tiles + kt);
          tma_load_2d_pair(&tmSB, bar, sf + Cfg::kSf, 0, 2 * nb * a.sf_tiles + kt);
          tma_load_2d_pair(&tmSB, bar, sf + 2 * Cfg::kSf, 0, (2 * nb + 1) * a.sf_tiles + kt);
        }
        __syncwarp();
        armed |= 1u << stage;
        parity = (parity & ~(1u << stage)) | (phase << stage);
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    // The stages' last uses are over, too: the leader's commits arrive here, and
    // this CTA must not end before the last of them has.
    for (int s = 0; s < kStages && ok; ++s) {
      ok = mbar_wait_warp(&empty[stage], phase ^ 1u, abort_flag, a.timeout_ns);
      if (++stage == kStages) {
        stage = 0;
        phase ^= 1u;
      }
    }
    if (!ok) {
      if (lane == 0)
        raise_abort(a.status, abort_flag, kStatusTimeoutBase | (kRoleProducer << 4) | 3);
      if (leader) {
        for (int s = 0; s < kStages; ++s)
          if (armed & (1u << s))
            (void)mbar_wait(&full[s], (parity >> s) & 1u, nullptr, a.timeout_ns);
      } else {
        // this CTA's loads complete on the leader's barriers, which it cannot
        // poll; give loads already issued ample time to land
        spin_ns(2000000);
      }
      __syncwarp();
    }
  } else if (warp == 1) {
    // ------------------------------------------------- MMA issuer (leader) ---
    if (leader) {
      const uint32_t base = __shfl_sync(0xffffffffu, tmem, 0);
      int stage = 0;
      uint32_t phase = 0, down = 0;
      int buf = 0;
      uint32_t acc_phase = 0, shared_phase = 0;
      bool ok = true;
      int site = 0;
      for (int tile = pair; tile < num_tiles && ok; tile += npairs, down ^= 1u) {
        ok = mbar_wait_warp(&acc_empty[buf], acc_phase ^ 1u, abort_flag, a.timeout_ns);
        if (!ok) {
          site = 5;
          break;
        }
        if (tile != pair) {  // the previous tile's epilogue has read the shared columns
          ok = mbar_wait_warp(shared_empty, shared_phase, abort_flag, a.timeout_ns);
          if (!ok) {
            site = 7;
            break;
          }
          shared_phase ^= 1u;
        }
        tc_fence_after_sync();
        const uint32_t d = base + static_cast<uint32_t>(buf ? Cfg::kAcc1 : 0);
        for (int i = 0; i < a.num_kb; ++i) {
          const int kb = down ? a.num_kb - 1 - i : i;
          ok = mbar_wait_warp(&full[stage], phase, abort_flag, a.timeout_ns);
          if (!ok) {
            site = 6;
            break;
          }
          tc_fence_after_sync();
          if (elect_one()) {
            const uint32_t s_addr = smem_u32(smS + stage * 3 * Cfg::kSf);
            // columns: 4 per tile of A's scales, then 8 per tile of B's (256 rows)
            const uint32_t sfa = base + Cfg::kSfBase + static_cast<uint32_t>(stage * Cfg::kSetCols);
            const uint32_t sfb = sfa + Kind<FMT>::kSfCols;
#pragma unroll
            for (int t = 0; t < Kind<FMT>::kSfTiles; ++t) {
              copy_scales<2>(sfa + 4 * t, (s_addr + t * kTileBytes) >> 4);
              copy_scales<2>(sfb + 8 * t, (s_addr + Cfg::kSf + t * kTileBytes) >> 4);
              copy_scales<2>(sfb + 8 * t + 4, (s_addr + 2 * Cfg::kSf + t * kTileBytes) >> 4);
            }
            issue_mmas<FMT, 2, kTile, kTile, 8>(d, smem_u32(smA + stage * Cfg::kOperand),
                                                smem_u32(smB + stage * Cfg::kOperand), sfa, sfb,
                                                a.row_bytes - kb * kRowBytes, i != 0);
            umma_commit_pair(&empty[stage], 0x3);  // stage free in both CTAs
            if (i == a.num_kb - 1) umma_commit_pair(&acc_full[buf], 0x3);  // both epilogues may read
          }
          __syncwarp();
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        buf ^= 1;
        if (buf == 0) acc_phase ^= 1u;
      }
      if (!ok) {
        if (elect_one()) {
          raise_abort(a.status, abort_flag, kStatusTimeoutBase | (kRoleMma << 4) | site);
          umma_commit_pair(drain, 0x1);
          (void)mbar_wait(drain, 0, nullptr, a.timeout_ns);
        }
        __syncwarp();
      }
    }
  } else {
    // ------------------------------------------------ epilogue (both CTAs) ---
    const int q = warp & 3;
    const int ew = warp - 2;
    const int g = ew >> 2;  // columns 64 g .. 64 g + 63 of the tile
    const uint64_t policy = l2_policy_evict_first();
    int buf = 0;
    uint32_t acc_phase = 0;
    for (int tile = pair; tile < num_tiles; tile += npairs) {
      int mb, nb;
      tile_coords(tile, num_m, num_n, a.group_m, mb, nb);
      int ok = 1;
      if (lane == 0) ok = mbar_wait(&acc_full[buf], acc_phase, abort_flag, a.timeout_ns) ? 1 : 0;
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) {
        if (lane == 0)
          raise_abort(a.status, abort_flag, kStatusTimeoutBase | (kRoleEpilogue << 4) | 3);
        break;
      }
      tc_fence_after_sync();
      const int row0 = mb * kTile + rank * kHalf + q * kWarpRows;
      const int col0 = nb * kTile + g * kWarpCols;
      uint32_t v[kWarpCols];
      tmem_load_32x32b_x64(tmem + (static_cast<uint32_t>(q * 32) << 16) +
                               static_cast<uint32_t>((buf ? Cfg::kAcc1 : 0) + g * kWarpCols),
                           v);
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        // the columns both buffers share: the last ones of buffer 0, the first of buffer 1
        const bool shares = buf == 0 ? (g + 1) * kWarpCols > Cfg::kAcc1
                                     : g * kWarpCols < Cfg::kOverlap;
        // Only where a later tile's MMAs wait for it: nothing else would keep
        // the leader from ending before an arrival of the other CTA lands.
        // (1500 x 2000 x 2000 MXFP4 7.86 us; 8.29 with every arrival and a
        // closing barrier that releases, 7.72 without either.)
        if (shares && tile + npairs < num_tiles) mbar_arrive_cluster_relaxed(shared_empty_leader);
        if (tile + 2 * npairs < num_tiles) mbar_arrive_cluster_relaxed(acc_empty_leader + buf * 8);
      }
      store_columns<T, ACT>(v, a, row0 + lane, col0, policy);
      buf ^= 1;
      if (buf == 0) acc_phase ^= 1u;
    }
  }

  tc_fence_before_sync();
  // No CTA of the pair frees TMEM while the other may still use it.  (A relaxed
  // arrival: every signal that the epilogues send to the leader's barriers has
  // been waited for by its MMA warp, and every commit of its to the other CTA's
  // by that CTA's producer and epilogue.)
  __syncwarp();
  cluster_arrive_relaxed();
  cluster_wait();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after_sync();
    tmem_dealloc_pair(tmem, 512);
  }
}

template <int FMT, class T, int ACT>
int launch(const MxGemmProblem& p, const DeviceCtx& d) {
  using Cfg = PairCfg<FMT>;
  static std::atomic<uint64_t> attr_done{0};
  static std::atomic<int> max_pairs[64] = {};  // resident pairs, per device (0 = not asked yet)
  auto kern = pair_gemm_kernel<FMT, T, ACT>;
  if (!ensure_smem_attr(reinterpret_cast<const void*>(kern), Cfg::kSmemBytes, d.device, attr_done))
    return runtime_error();
  const int64_t row_bytes = mx_row_bytes(p.K, FMT);
  const int64_t sf_tiles = scale_tiles(p.K);
  constexpr int kBox = Kind<FMT>::kSfTiles;
  CUtensorMap tA, tB, tSA, tSB;
  int rc = encode_tmap_u8_2d(&tA, p.A, row_bytes, p.M, p.lda, kHalf);
  if (rc == 0) rc = encode_tmap_u8_2d(&tB, p.B, row_bytes, p.N, p.ldb, kHalf);
  if (rc == 0) rc = encode_tmap_scales(&tSA, p.SA, (p.M + 127) / 128 * sf_tiles, kBox);
  if (rc == 0) rc = encode_tmap_scales(&tSB, p.SB, (p.N + 127) / 128 * sf_tiles, kBox);
  if (rc != 0) return rc;
  Launch l(dim3(2 * (d.sm_count / 2)), dim3(kThreads), Cfg::kSmemBytes, p.stream);
  l.cluster(2);
  int resident = max_pairs[d.device & 63].load(std::memory_order_relaxed);
  if (resident == 0) {
    if (cudaOccupancyMaxActiveClusters(&resident, kern, &l.cfg) != cudaSuccess || resident <= 0) {
      cudaGetLastError();
      resident = d.sm_count / 2;
    }
    max_pairs[d.device & 63].store(resident, std::memory_order_relaxed);
  }
  const int64_t tiles = ((p.M + kTile - 1) / kTile) * ((p.N + kTile - 1) / kTile);
  if (tiles > INT32_MAX) return GEMM_ERR_INVALID_ARG;
  l.cfg.gridDim = dim3(2u * static_cast<unsigned>(tiles < resident ? tiles : resident));
  const PairArgs a{static_cast<uint16_t*>(p.C),
                   static_cast<const uint16_t*>(p.bias),
                   p.ldc,
                   static_cast<int>(p.M),
                   static_cast<int>(p.N),
                   static_cast<int>(row_bytes),
                   static_cast<int>(sf_tiles),
                   static_cast<int>((row_bytes + kRowBytes - 1) / kRowBytes),
                   group_tiles(kPanelRows, kTile, kTile),
                   (reinterpret_cast<uintptr_t>(p.C) & 31) == 0 && p.ldc % 16 == 0,
                   d.status,
                   d.timeout_ns};
  const cudaError_t e = cudaLaunchKernelEx(&l.cfg, kern, tA, tB, tSA, tSB, a);
  return launched(e);
}

template <int FMT, class T>
int launch_act(const MxGemmProblem& p, const DeviceCtx& d) {
  switch (p.act) {
    case kActRelu: return launch<FMT, T, kActRelu>(p, d);
    case kActGelu: return launch<FMT, T, kActGelu>(p, d);
    default: return launch<FMT, T, kActNone>(p, d);
  }
}

}  // namespace

int launch_mx_pair_gemm(const MxGemmProblem& p, const DeviceCtx& d) {
  if (p.format == MX_FP8)
    return p.dtype == MX_F16 ? launch_act<MX_FP8, __half>(p, d)
                             : launch_act<MX_FP8, __nv_bfloat16>(p, d);
  return p.dtype == MX_F16 ? launch_act<MX_FP4, __half>(p, d)
                           : launch_act<MX_FP4, __nv_bfloat16>(p, d);
}

}  // namespace mx
}  // namespace ttc
