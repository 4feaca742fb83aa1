// C = act(A B^T + bias) for MX operands, middling shapes: swap-AB tiles of 256
// rows of B by 128 rows of A for a CTA pair, with K split over a cluster of
// pairs.
//
// The split kernel's tile (mx_gemm_split.cu) takes 192 bytes of each row pair of
// K for 64 x 128 products.  From 65 rows of A on, an SM of a pair stages 128 rows
// of B and 64 of A and computes 128 x 128 products from them and the other SM's
// half of A: half the bytes a product.  The rest is as there: every CTA leaves
// its fp32 part (128 rows of A by its 128 rows of B) in its shared memory, sends
// the rows of A that another part's CTA finishes to it, and adds what it
// receives in the order of the parts.  256 x 4096 x 8192 MXFP8: 14.1 us, 19.7
// in the split kernel.  Of 20,500 cycles the first load takes 2,400, the k-blocks
// 13,600 (60 bytes a cycle into an SM), the accumulator's way to shared memory
// 700, the sending 2,300 and the last rows 1,400; sending and finishing in
// halves changes nothing.
#include "mx_umma.cuh"
#include "tile_common.cuh"

namespace ttc {
namespace mx {
namespace {

constexpr int kTileN = 256;   // rows of B per pair
constexpr int kHalfN = 128;   // and per CTA
constexpr int kTileM = 128;   // rows of A per pair
constexpr int kHalfM = 64;    // of which a CTA stages
constexpr int kMaxParts = 4;  // pairs of a cluster
constexpr int kStages = 8;
constexpr int kEpiWarps = 8;  // two per TMEM lane quarter, 64 rows of A each
constexpr int kThreads = 64 + 32 * kEpiWarps;

template <int FMT>
struct Cfg {
  static constexpr int kWBytes = kHalfN * kRowBytes;
  static constexpr int kXBytes = kHalfM * kRowBytes;
  static constexpr int kSf = Kind<FMT>::kSfTiles * kTileBytes;  // scales of 128 rows
  static constexpr int kStageBytes = kWBytes + kXBytes + 2 * kSf;
  static constexpr int kRing = kStages * kStageBytes;
  static constexpr int kPartBytes = kTileM * kHalfN * 4;
  static constexpr int kSmemBytes = 1024 + kRing + (2 * kStages + 3) * 8 + 16;
  // accumulator, then one set of scales per stage: a stage's columns are
  // written again only after the MMAs that read them have completed
  static constexpr int kSetCols = 2 * Kind<FMT>::kSfCols;
  static constexpr uint32_t kTmemCols = 256;
  static_assert(kTileM + kStages * kSetCols <= 256, "TMEM columns");
  static_assert(kPartBytes + slot_rows(kTileM, kMaxParts) * kHalfN * 4 <= kRing, "parts");
  static_assert(kSmemBytes <= kMaxDynamicSmem, "shared memory budget");
};

struct Args {
  Output out;
  int row_bytes, sf_tiles, num_kb, tiles_m;
  int* status;
  uint64_t timeout_ns;
};

template <int FMT>
__global__ void __launch_bounds__(kThreads, 1)
    pair_split_gemm_kernel(const __grid_constant__ CUtensorMap tmB,
                           const __grid_constant__ CUtensorMap tmA,
                           const __grid_constant__ CUtensorMap tmSB,
                           const __grid_constant__ CUtensorMap tmSA, const Args a) {
  using C = Cfg<FMT>;
  constexpr int kSfTiles = Kind<FMT>::kSfTiles;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* smW = smem;
  uint8_t* smX = smW + kStages * C::kWBytes;
  uint8_t* smS = smX + kStages * C::kXBytes;  // per stage: scales of B, scales of A
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kRing);
  uint64_t* empty = full + kStages;
  uint64_t* acc_full = empty + kStages;
  uint64_t* drain = acc_full + 1;
  uint64_t* received = drain + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(received + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);  // uniform
  const int lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const int parts = static_cast<int>(cluster_size()) / 2;
  const int part = rank >> 1, half = rank & 1;
  const bool leader = half == 0;
  const uint16_t pair_mask = static_cast<uint16_t>(0x3 << (rank & ~1));
  const int tile = static_cast<int>(cluster_id_x());
  const int mt = tile % a.tiles_m, nt = tile / a.tiles_m;
  const int m0 = mt * kTileM, n0 = nt * kTileN + half * kHalfN;
  const int rows = min(kTileM, a.out.M - m0);
  const int kb_begin = static_cast<int>(static_cast<int64_t>(a.num_kb) * part / parts);
  const int kb_end = static_cast<int>(static_cast<int64_t>(a.num_kb) * (part + 1) / parts);
  // the rows of A that part r finishes are [first_row(r), first_row(r + 1))
  auto first_row = [&](int r) { return rows * r / parts; };
  const int r0 = first_row(part), r1 = first_row(part + 1);
  const int slot_bytes = (kTileM + parts - 1) / parts * kHalfN * 4;

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
    tma_prefetch_desc(&tmSB);
    tma_prefetch_desc(&tmSA);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, C::kTmemCols);
    tmem_relinquish_alloc_permit_pair();
  }
  tc_fence_before_sync();
  cluster_sync();  // barriers initialised, TMEM of both SMs of the pair allocated
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  grid_dependency_trigger();
  grid_dependency_wait();
  const int c = static_cast<int>(threadIdx.x & 15) * 8;  // the columns this thread finishes
  const uint4 bias = load_bias(a.out, n0 + c);

  if (warp == 0) {
    // --------------------------------------------- TMA producer (every CTA) ---
    int stage = 0;
    uint32_t phase = 0, armed = 0, parity = 0;
    bool ok = true;
    const uint32_t full_leader = map_to_cta(smem_u32(full), static_cast<uint32_t>(rank & ~1));
    for (int kb = kb_begin; kb < kb_end; ++kb) {
      ok = mbar_wait_warp(&empty[stage], phase ^ 1u, abort_flag, a.timeout_ns);
      if (!ok) break;
      if (elect_one()) {
        if (leader) mbar_arrive_expect_tx(&full[stage], 2 * C::kStageBytes);
        const uint32_t bar = full_leader + stage * 8;
        const int kt = kb * kSfTiles;
        uint8_t* sf = smS + stage * 2 * C::kSf;
        tma_load_2d_pair(&tmB, bar, smW + stage * C::kWBytes, kb * kRowBytes, n0);
        tma_load_2d_pair(&tmA, bar, smX + stage * C::kXBytes, kb * kRowBytes, m0 + half * kHalfM);
        // past the last row of tiles these read another row's or zeros: what
        // they scale is not stored
        tma_load_2d_pair(&tmSB, bar, sf, 0, (2 * nt + half) * a.sf_tiles + kt);
        tma_load_2d_pair(&tmSA, bar, sf + C::kSf, 0, mt * a.sf_tiles + kt);
      }
      __syncwarp();
      armed |= 1u << stage;
      parity = (parity & ~(1u << stage)) | (phase << stage);
      if (++stage == kStages) {
        stage = 0;
        phase ^= 1u;
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
        raise_abort(a.status, abort_flag, kStatusTimeoutBase | (kRoleProducer << 4) | 4);
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
    cluster_arrive_relaxed();
  } else if (warp == 1) {
    // ------------------------------------------- MMA issuer (pair leaders) ---
    if (leader) {
      const uint32_t base = __shfl_sync(0xffffffffu, tmem, 0);
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int kb = kb_begin; kb < kb_end; ++kb) {
        ok = mbar_wait_warp(&full[stage], phase, abort_flag, a.timeout_ns);
        if (!ok) break;
        tc_fence_after_sync();
        if (elect_one()) {
          const uint32_t s_addr = smem_u32(smS + stage * 2 * C::kSf);
          const uint32_t sfw = base + kTileM + static_cast<uint32_t>(stage * C::kSetCols);
          const uint32_t sfx = sfw + Kind<FMT>::kSfCols;
#pragma unroll
          for (int t = 0; t < kSfTiles; ++t) {
            copy_scales<2>(sfw + 4 * t, (s_addr + t * kTileBytes) >> 4);
            copy_scales<2>(sfx + 4 * t, (s_addr + C::kSf + t * kTileBytes) >> 4);
          }
          issue_mmas<FMT, 2, kTileN, kTileM, 4>(base, smem_u32(smW + stage * C::kWBytes),
                                                smem_u32(smX + stage * C::kXBytes), sfw, sfx,
                                                a.row_bytes - kb * kRowBytes, kb != kb_begin);
          umma_commit_pair(&empty[stage], pair_mask);
          if (kb == kb_end - 1) umma_commit_pair(acc_full, pair_mask);
        }
        __syncwarp();
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (!ok) {
        if (elect_one()) {
          raise_abort(a.status, abort_flag, kStatusTimeoutBase | (kRoleMma << 4) | 9);
          umma_commit_pair(drain, static_cast<uint16_t>(1 << rank));
          (void)mbar_wait(drain, 0, nullptr, a.timeout_ns);
        }
        __syncwarp();
      }
    }
    __syncwarp();
    cluster_arrive_relaxed();
  } else {
    // -------------------------------- accumulator to shared memory (every CTA) ---
    int ok = 1;
    if (lane == 0) ok = mbar_wait(acc_full, 0, abort_flag, a.timeout_ns) ? 1 : 0;
    ok = __shfl_sync(0xffffffffu, ok, 0);
    // all loads of the pair have landed and all its MMAs have read them: the
    // ring is free, for what others send, too
    cluster_arrive_relaxed();
    if (ok) {
      tc_fence_after_sync();
      const int q = warp & 3, g = (warp - 2) >> 2;
      float* mine = reinterpret_cast<float*>(smem) + q * 32 + lane;
#pragma unroll 1
      for (int r = g * 64; r < g * 64 + 64; r += 32) {
        if (r >= rows) break;
        uint32_t v[32];
        tmem_load_32x32b_x32(tmem + (static_cast<uint32_t>(q * 32) << 16) + r, v);
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (r + i < rows) mine[(r + i) * kHalfN] = __uint_as_float(v[i]);
      }
    } else if (lane == 0) {
      raise_abort(a.status, abort_flag, kStatusTimeoutBase | (kRoleEpilogue << 4) | 4);
    }
  }
  __syncwarp();
  tc_fence_before_sync();
  fence_proxy_async_smem();  // the part is read by bulk copies
  __syncthreads();           // all of this CTA's part is written
  cluster_wait();            // all rings are free
  uint8_t* incoming = smem + C::kPartBytes;
  if (parts > 1) {
    if (threadIdx.x == 0) {
      mbar_arrive_expect_tx(received,
                            static_cast<uint32_t>((parts - 1) * (r1 - r0) * kHalfN * 4));
      for (int k = 1; k < parts && *abort_flag == 0; ++k) {
        const int to = part + k < parts ? part + k : part + k - parts;
        const int from_row = first_row(to), n = first_row(to + 1) - from_row;
        if (n == 0) continue;
        // the receiver keeps its slots in the order of the parts, without its own
        const int slot = part < to ? part : part - 1;
        const uint32_t cta = static_cast<uint32_t>(2 * to + half);
        bulk_push(map_to_cta(smem_u32(incoming) + static_cast<uint32_t>(slot * slot_bytes), cta),
                  smem + from_row * kHalfN * 4, static_cast<uint32_t>(n * kHalfN * 4),
                  map_to_cta(smem_u32(received), cta));
      }
    }
    // (after an abort, too: what others have sent has to land before this CTA ends)
    if (r1 > r0 && !mbar_wait(received, 0, nullptr, a.timeout_ns))
      raise_abort(a.status, abort_flag, kStatusTimeoutBase | (kRoleEpilogue << 4) | 2);
  }
  __syncwarp();
  cluster_arrive_relaxed();  // what was sent to this CTA has left the others' shared memory
  if (*abort_flag == 0)
    finish_rows<kThreads>(a.out, m0 + r0, n0 + c, r1 - r0, bias, parts, [&](int s) {
      return reinterpret_cast<const float*>(
                 s == part ? smem + r0 * kHalfN * 4
                           : incoming + (s < part ? s : s - 1) * slot_bytes) + c;
    });
  __syncwarp();
  // no CTA leaves while its copies may still read its shared memory (the
  // leader's commits have been waited for by producers and epilogues)
  cluster_wait();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc_pair(tmem, C::kTmemCols);
  }
}

template <int FMT>
int launch(const MxGemmProblem& p, const DeviceCtx& d) {
  using C = Cfg<FMT>;
  static std::atomic<uint64_t> attr_done{0};
  static Residency residency[64];
  auto kern = pair_split_gemm_kernel<FMT>;
  if (!ensure_smem_attr(reinterpret_cast<const void*>(kern), C::kSmemBytes, d.device, attr_done))
    return runtime_error();
  const int64_t row_bytes = mx_row_bytes(p.K, FMT);
  const int64_t sf_tiles = scale_tiles(p.K);
  const int64_t num_kb = (row_bytes + kRowBytes - 1) / kRowBytes;
  const int64_t tiles_m = (p.M + kTileM - 1) / kTileM;
  const int64_t tiles = tiles_m * ((p.N + kTileN - 1) / kTileN);
  // as many parts of at least four k-blocks as run in one wave
  int parts = 1;
  for (int s = 2; s <= kMaxParts && num_kb >= 4 * s; ++s)
    if (tiles <= residency[d.device & 63].of(2 * s, kern, kThreads, C::kSmemBytes, d)) parts = s;
  if (2 * parts * tiles > INT32_MAX) return GEMM_ERR_INVALID_ARG;
  constexpr int kBox = Kind<FMT>::kSfTiles;
  CUtensorMap tB, tA, tSB, tSA;
  int rc = encode_tmap_u8_2d(&tB, p.B, row_bytes, p.N, p.ldb, kHalfN);
  if (rc == 0) rc = encode_tmap_u8_2d(&tA, p.A, row_bytes, p.M, p.lda, kHalfM);
  if (rc == 0) rc = encode_tmap_scales(&tSB, p.SB, (p.N + 127) / 128 * sf_tiles, kBox);
  if (rc == 0) rc = encode_tmap_scales(&tSA, p.SA, (p.M + 127) / 128 * sf_tiles, kBox);
  if (rc != 0) return rc;
  Launch l(dim3(static_cast<unsigned>(2 * parts * tiles)), dim3(kThreads), C::kSmemBytes, p.stream);
  l.cluster(static_cast<unsigned>(2 * parts));
  const Args a{output_of(p),
               static_cast<int>(row_bytes),
               static_cast<int>(sf_tiles),
               static_cast<int>(num_kb),
               static_cast<int>(tiles_m),
               d.status,
               d.timeout_ns};
  const cudaError_t e = cudaLaunchKernelEx(&l.cfg, kern, tB, tA, tSB, tSA, a);
  return launched(e);
}

}  // namespace

int launch_mx_pair_split_gemm(const MxGemmProblem& p, const DeviceCtx& d) {
  return p.format == MX_FP8 ? launch<MX_FP8>(p, d) : launch<MX_FP4>(p, d);
}

}  // namespace mx
}  // namespace ttc
