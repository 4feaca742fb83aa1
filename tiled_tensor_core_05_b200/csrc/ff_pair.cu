// 16-bit products of large shapes: a CTA pair per 256 x 256 tile, persistent,
// tcgen05.mma.cta_group::2.  One main loop serves three forms (ff_internal.h):
//
//   gated    the tile's columns are 128 of the gate's and the same 128 of the other
//            projection: CTA 0 of the pair stages rows of Wg, CTA 1 of Wu, and each
//            accumulator row holds both, so that act(gate) * up needs nothing from
//            another thread and the projections never leave the SM
//   concat   dX = dG Wg + dU Wu: one sum over 2 F elements, the k-blocks of the
//            first pair of operands followed by those of the second
//   stack    dWg and dWu: two products of one size, their tiles one after the other
//
//   warp 0     TMA producer of each CTA: 64 elements of K of 128 rows of A and 128
//              rows of B per k-block, K-major or (stored K x M, K x N) MN-major,
//              128-byte swizzle, 7 stages
//   warp 1     TMEM; the leader issues the MMAs of both SMs
//   warps 2-17 two accumulators of 256 columns, the epilogue of one beside the MMAs
//              of the other
//
// Every other wave sweeps K downwards, so that it starts on what the wave before has
// left in L2, as in gemm_tile.cu.
#include "ff_common.cuh"
#include "tile_common.cuh"

namespace ttc {
namespace ff {
namespace {

using mx::elect_one;
using mx::mbar_wait_warp;

constexpr int kTile = 256;     // rows and columns of a pair's tile
constexpr int kHalf = 128;     // rows of A and of B per CTA
constexpr int kBK = 64;        // elements of K per k-block
constexpr int kStages = 7;
constexpr int kOperand = kHalf * kBK * 2;  // bytes of A, and of B, per stage
constexpr int kStageBytes = 2 * kOperand;
constexpr int kSlab = kBK * 64 * 2;  // 64 rows of an MN-major operand
constexpr int kEpiWarps = 16;        // four per TMEM lane quarter, 64 columns each
constexpr int kWarpCols = 64;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kPanelRows = 4096;  // rows of A per raster panel
constexpr int kBars = 2 * kStages + 5;
constexpr int kSmemBytes = 1024 + kStages * kStageBytes + kBars * 8 + 16;
static_assert(kSmemBytes <= kMaxDynamicSmem, "shared memory budget");

struct PairArgs {
  uint16_t* C[2];
  int64_t ldc[2];
  float *gate, *up;
  int64_t ld_gate, ld_up;
  int M, N;         // rows and columns of an output
  int cols;         // columns of an output per tile: 256, or 128 of the gated form
  int num_kb;       // k-blocks of a tile
  int source_kb;    // of which the first operands' (concat; else num_kb)
  int problem_tiles;  // tiles of an output (stack: the second output's follow)
  int num_tiles;
  int group_m;
  int a_mn, b_mn;   // stored K x M, K x N
  int b_step;       // rows of B between the CTAs of a pair: 128, gated 0
  uint32_t idesc;
  int wide;         // rows of the outputs start on 32 bytes
  int* status;
  uint64_t timeout_ns;
};

// Instruction descriptor of kind::f16 (sm100.cuh), fp16 or bf16 operands.
uint32_t pair_idesc(int dtype, bool a_mn, bool b_mn) {
  const uint32_t type = dtype == MX_BF16 ? (1u << 7) | (1u << 10) : 0u;
  return idesc_f16_f32(kTile, kTile, a_mn, b_mn) | type;
}

// 32 aligned bytes, written once and not read again here.
__device__ __forceinline__ void store_32(void* p, const uint32_t (&h)[8], uint64_t policy) {
  asm volatile(
      "st.global.L2::cache_hint.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8}, %9;" ::"l"(p),
      "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3]), "r"(h[4]), "r"(h[5]), "r"(h[6]), "r"(h[7]),
      "l"(policy)
      : "memory");
}

// 16 columns of a row as 16-bit values, of which n exist.
__device__ __forceinline__ void store_16(uint16_t* p, const uint32_t (&h)[8], int n, int wide,
                                         uint64_t policy) {
  if (n >= 16 && wide) {
    store_32(p, h, policy);
  } else {
    mx::store8(p, make_uint4(h[0], h[1], h[2], h[3]), n);
    if (n > 8) mx::store8(p + 8, make_uint4(h[4], h[5], h[6], h[7]), n - 8);
  }
}

// 8 fp32 columns of a row.
__device__ __forceinline__ void store_f32(float* p, const uint32_t* v, int n, int wide,
                                          uint64_t policy) {
  if (n >= 8 && wide) {
    uint32_t h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = v[i];
    store_32(p, h, policy);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = __uint_as_float(v[i]);
  }
}

// 64 accumulators of this thread's row of C, rounded.
template <class T>
__device__ __forceinline__ void store_plain(const uint32_t (&v)[kWarpCols], const PairArgs& a,
                                            int p, int row, int col0, uint64_t policy) {
  if (row >= a.M) return;
  uint16_t* c = a.C[p] + row * a.ldc[p] + col0;
#pragma unroll
  for (int i = 0; i < kWarpCols; i += 16) {
    const int n = a.N - (col0 + i);
    if (n <= 0) break;
    uint32_t h[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      h[k] = mx::pack2<T>(__uint_as_float(v[i + 2 * k]), __uint_as_float(v[i + 2 * k + 1]));
    store_16(c + i, h, n, a.wide, policy);
  }
}

// 32 columns of this thread's row of H: gate sums in v[0..31], the others in v[32..63].
template <class T, int ACT>
__device__ __forceinline__ void store_gated(const uint32_t (&v)[kWarpCols], const PairArgs& a,
                                            int row, int col0, uint64_t policy) {
  if (row >= a.M) return;
  const int left = a.N - col0;
  if (left <= 0) return;
  if (a.gate != nullptr) {
    float* g = a.gate + row * a.ld_gate + col0;
    float* u = a.up + row * a.ld_up + col0;
#pragma unroll
    for (int i = 0; i < 32; i += 8) {
      if (i >= left) break;
      store_f32(g + i, &v[i], left - i, a.wide, policy);
      store_f32(u + i, &v[32 + i], left - i, a.wide, policy);
    }
  }
  uint16_t* c = a.C[0] + row * a.ldc[0] + col0;
#pragma unroll
  for (int i = 0; i < 32; i += 16) {
    if (i >= left) break;
    uint32_t h[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int j = i + 2 * k;
      const float2 x = __fmul2_rn(
          ff_activate2<ACT>(make_float2(__uint_as_float(v[j]), __uint_as_float(v[j + 1]))),
          make_float2(__uint_as_float(v[32 + j]), __uint_as_float(v[33 + j])));
      h[k] = mx::pack2<T>(x.x, x.y);
    }
    store_16(c + i, h, left - i, a.wide, policy);
  }
}

// 32 lanes x 32 columns at two places of TMEM (one wait, see sm100.cuh).
__device__ __forceinline__ void tmem_load_two_x32(uint32_t first, uint32_t second,
                                                  uint32_t (&r)[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%64];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%65];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
        "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]),
        "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]),
        "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]), "=r"(r[49]),
        "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
        "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]),
        "=r"(r[62]), "=r"(r[63])
      : "r"(first), "r"(second)
      : "memory");
}

// D[tmem] (+)= A B of a pair; a, b: low descriptor words (mx_umma.cuh).
__device__ __forceinline__ void pair_mma(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tmov.b64 da, {%1, %5};\n\t"
      "mov.b64 db, {%2, %5};\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], da, db, %3, p;\n\t}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "r"(mx::kDescHigh)
      : "memory");
}

// GATED_ACT: the activation of the gated form, or -1 for the plain ones.
template <class T, int GATED_ACT>
__global__ void __launch_bounds__(kThreads, 1)
    ff_pair_kernel(const __grid_constant__ CUtensorMap tmA0,
                   const __grid_constant__ CUtensorMap tmA1,
                   const __grid_constant__ CUtensorMap tmB0,
                   const __grid_constant__ CUtensorMap tmB1, const PairArgs a) {
  constexpr bool kGatedForm = GATED_ACT >= 0;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* smA = smem;
  uint8_t* smB = smA + kStages * kOperand;
  uint64_t* full = reinterpret_cast<uint64_t*>(smB + kStages * kOperand);
  uint64_t* empty = full + kStages;
  uint64_t* acc_full = empty + kStages;  // [2]
  uint64_t* acc_empty = acc_full + 2;    // [2] a buffer has been read
  uint64_t* drain = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(full + kBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);  // uniform
  const int lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const bool leader = rank == 0;
  const int pair = static_cast<int>(cluster_id_x());
  const int npairs = static_cast<int>(num_clusters_x());
  const int num_m = (a.M + kTile - 1) / kTile;
  const int num_n = (a.N + a.cols - 1) / a.cols;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 2 * kEpiWarps);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmA0);
    tma_prefetch_desc(&tmA1);
    tma_prefetch_desc(&tmB0);
    tma_prefetch_desc(&tmB1);
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

  // a tile's output and place
  auto place = [&](int tile, int& p, int& mb, int& nb) {
    p = tile >= a.problem_tiles ? 1 : 0;
    tile_coords(tile - p * a.problem_tiles, num_m, num_n, a.group_m, mb, nb);
  };

  if (warp == 0) {
    // --------------------------------------------- TMA producer (both CTAs) ---
    int stage = 0;
    uint32_t phase = 0, armed = 0, parity = 0, down = 0;
    bool ok = true;
    for (int tile = pair; tile < a.num_tiles && ok; tile += npairs, down ^= 1u) {
      int p, mb, nb;
      place(tile, p, mb, nb);
      const int a_row = mb * kTile + rank * kHalf;
      const int b_row = nb * a.cols + rank * a.b_step;
      for (int i = 0; i < a.num_kb; ++i) {
        int kb = down ? a.num_kb - 1 - i : i;
        ok = mbar_wait_warp(&empty[stage], phase ^ 1u, abort_flag, a.timeout_ns);
        if (!ok) break;
        if (elect_one()) {
          if (leader) mbar_arrive_expect_tx(&full[stage], 2 * kStageBytes);
          const uint32_t bar = full_leader + stage * 8;
          const bool second = kb >= a.source_kb;
          if (second) kb -= a.source_kb;
          const CUtensorMap* tA = second || p ? &tmA1 : &tmA0;
          const CUtensorMap* tB = second || (kGatedForm && rank) ? &tmB1 : &tmB0;
          uint8_t* sa = smA + stage * kOperand;
          uint8_t* sb = smB + stage * kOperand;
          if (!a.a_mn) {
            tma_load_2d_pair(tA, bar, sa, kb * kBK, a_row);
          } else {
            tma_load_2d_pair(tA, bar, sa, a_row, kb * kBK);
            tma_load_2d_pair(tA, bar, sa + kSlab, a_row + 64, kb * kBK);
          }
          if (!a.b_mn) {
            tma_load_2d_pair(tB, bar, sb, kb * kBK, b_row);
          } else {
            tma_load_2d_pair(tB, bar, sb, b_row, kb * kBK);
            tma_load_2d_pair(tB, bar, sb + kSlab, b_row + 64, kb * kBK);
          }
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
      // low descriptor words: leading dimension (slabs of an MN-major operand),
      // and what 16 elements of K add to the address
      const uint32_t a_lead = a.a_mn ? (kSlab >> 4) << 16 : 1u << 16;
      const uint32_t b_lead = a.b_mn ? (kSlab >> 4) << 16 : 1u << 16;
      const uint32_t a_step = a.a_mn ? (16 * 128) >> 4 : (16 * 2) >> 4;
      const uint32_t b_step = a.b_mn ? (16 * 128) >> 4 : (16 * 2) >> 4;
      int stage = 0;
      uint32_t phase = 0;
      int buf = 0;
      uint32_t acc_phase = 0;
      bool ok = true;
      int site = 0;
      for (int tile = pair; tile < a.num_tiles && ok; tile += npairs) {
        ok = mbar_wait_warp(&acc_empty[buf], acc_phase ^ 1u, abort_flag, a.timeout_ns);
        if (!ok) {
          site = 5;
          break;
        }
        tc_fence_after_sync();
        const uint32_t d = base + static_cast<uint32_t>(buf * kTile);
        for (int i = 0; i < a.num_kb; ++i) {
          ok = mbar_wait_warp(&full[stage], phase, abort_flag, a.timeout_ns);
          if (!ok) {
            site = 6;
            break;
          }
          tc_fence_after_sync();
          if (elect_one()) {
            const uint32_t al = ((smem_u32(smA + stage * kOperand) >> 4) & 0x3FFFu) | a_lead;
            const uint32_t bl = ((smem_u32(smB + stage * kOperand) >> 4) & 0x3FFFu) | b_lead;
#pragma unroll
            for (int k = 0; k < kBK / 16; ++k)
              pair_mma(d, al + k * a_step, bl + k * b_step, a.idesc, (i | k) != 0 ? 1u : 0u);
            umma_commit_pair(&empty[stage], 0x3);  // stage free in both CTAs
            if (i == a.num_kb - 1) umma_commit_pair(&acc_full[buf], 0x3);  // both may read
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
    const int g = (warp - 2) >> 2;
    const uint64_t policy = l2_policy_evict_first();
    int buf = 0;
    uint32_t acc_phase = 0;
    for (int tile = pair; tile < a.num_tiles; tile += npairs) {
      int p, mb, nb;
      place(tile, p, mb, nb);
      int ok = 1;
      if (lane == 0) ok = mbar_wait(&acc_full[buf], acc_phase, abort_flag, a.timeout_ns) ? 1 : 0;
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) {
        if (lane == 0)
          raise_abort(a.status, abort_flag, kStatusTimeoutBase | (kRoleEpilogue << 4) | 3);
        break;
      }
      tc_fence_after_sync();
      const int row = mb * kTile + rank * kHalf + q * 32 + lane;
      const uint32_t t_row =
          tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(buf * kTile);
      uint32_t v[kWarpCols];
      if constexpr (kGatedForm)
        tmem_load_two_x32(t_row + g * 32, t_row + kHalf + g * 32, v);
      else
        tmem_load_32x32b_x64(t_row + g * kWarpCols, v);
      tc_fence_before_sync();
      __syncwarp();
      // only where a later tile's MMAs wait for it: nothing else would keep the
      // leader from ending before an arrival of the other CTA lands
      if (lane == 0 && tile + 2 * npairs < a.num_tiles)
        mbar_arrive_cluster_relaxed(acc_empty_leader + buf * 8);
      if constexpr (kGatedForm)
        store_gated<T, GATED_ACT>(v, a, row, nb * kHalf + g * 32, policy);
      else
        store_plain<T>(v, a, p, row, nb * kTile + g * kWarpCols, policy);
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
  mx::cluster_arrive_relaxed();
  mx::cluster_wait();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after_sync();
    tmem_dealloc_pair(tmem, 512);
  }
}

// The map of an operand of `rows` rows of K elements, or stored K x rows.
int encode_operand(CUtensorMap* map, const Mat& m, int64_t rows, int64_t K, bool mn) {
  if (mn) return encode_tmap_f16_2d(map, m.p, rows, K, m.ld, 64, kBK);
  return encode_tmap_f16_2d(map, m.p, K, rows, m.ld, kBK, kHalf);
}

bool on_32_bytes(const void* p, int64_t ld, int bytes) {
  return (reinterpret_cast<uintptr_t>(p) & 31) == 0 && ld * bytes % 32 == 0;
}

template <class T, int GATED_ACT>
int launch(const Product& p, const DeviceCtx& d) {
  static std::atomic<uint64_t> attr_done{0};
  static std::atomic<int> max_pairs[64] = {};  // resident pairs, per device (0 = not asked yet)
  auto kern = ff_pair_kernel<T, GATED_ACT>;
  if (!ensure_smem_attr(reinterpret_cast<const void*>(kern), kSmemBytes, d.device, attr_done))
    return runtime_error();
  const bool a_mn = p.form == kStack, b_mn = p.form != kGated;
  CUtensorMap tA[2], tB[2];
  for (int i = 0; i < 2; ++i) {
    // (a form with one operand of a kind names it twice)
    int rc = encode_operand(&tA[i], p.A[i], p.M, p.K, a_mn);
    if (rc == 0) rc = encode_operand(&tB[i], p.B[i], p.N, p.K, b_mn);
    if (rc != 0) return rc;
  }
  Launch l(dim3(2 * (d.sm_count / 2)), dim3(kThreads), kSmemBytes, p.stream);
  l.cluster(2);
  int resident = max_pairs[d.device & 63].load(std::memory_order_relaxed);
  if (resident == 0) {
    if (cudaOccupancyMaxActiveClusters(&resident, kern, &l.cfg) != cudaSuccess || resident <= 0) {
      cudaGetLastError();
      resident = d.sm_count / 2;
    }
    max_pairs[d.device & 63].store(resident, std::memory_order_relaxed);
  }
  const int cols = p.form == kGated ? kHalf : kTile;
  const int64_t problem_tiles = (p.M + kTile - 1) / kTile * ((p.N + cols - 1) / cols);
  const int64_t tiles = problem_tiles * (p.form == kStack ? 2 : 1);
  const int64_t blocks = (p.K + kBK - 1) / kBK;
  if (tiles > INT32_MAX / 2) return GEMM_ERR_INVALID_ARG;
  l.cfg.gridDim = dim3(2u * static_cast<unsigned>(tiles < resident ? tiles : resident));
  const int outputs = p.form == kStack ? 2 : 1;
  bool wide = true;
  for (int i = 0; i < outputs; ++i) wide = wide && on_32_bytes(p.C[i].p, p.C[i].ld, 2);
  if (p.gate != nullptr)
    wide = wide && on_32_bytes(p.gate, p.ld_gate, 4) && on_32_bytes(p.up, p.ld_up, 4);
  PairArgs a{};
  for (int i = 0; i < 2; ++i) {
    a.C[i] = static_cast<uint16_t*>(const_cast<void*>(p.C[i].p));
    a.ldc[i] = p.C[i].ld;
  }
  a.gate = p.gate;
  a.up = p.up;
  a.ld_gate = p.ld_gate;
  a.ld_up = p.ld_up;
  a.M = static_cast<int>(p.M);
  a.N = static_cast<int>(p.N);
  a.cols = cols;
  a.source_kb = static_cast<int>(blocks);
  a.num_kb = static_cast<int>(p.form == kConcat ? 2 * blocks : blocks);
  a.problem_tiles = static_cast<int>(problem_tiles);
  a.num_tiles = static_cast<int>(tiles);
  a.group_m = group_tiles(kPanelRows, kTile, kTile);
  a.a_mn = a_mn;
  a.b_mn = b_mn;
  a.b_step = p.form == kGated ? 0 : kHalf;
  a.idesc = pair_idesc(p.dtype, a_mn, b_mn);
  a.wide = wide;
  a.status = d.status;
  a.timeout_ns = d.timeout_ns;
  return launched(cudaLaunchKernelEx(&l.cfg, kern, tA[0], tA[1], tB[0], tB[1], a));
}

template <class T>
int launch_form(const Product& p, const DeviceCtx& d) {
  if (p.form != kGated) return launch<T, -1>(p, d);
  switch (p.act) {
    case kActSilu: return launch<T, kActSilu>(p, d);
    case kActGelu: return launch<T, kActGelu>(p, d);
    case kActRelu: return launch<T, kActRelu>(p, d);
    default: return launch<T, kActNone>(p, d);
  }
}

}  // namespace

int launch_pair_product(const Product& p, const DeviceCtx& d) {
  return p.dtype == MX_F16 ? launch_form<__half>(p, d) : launch_form<__nv_bfloat16>(p, d);
}

}  // namespace ff
}  // namespace ttc
