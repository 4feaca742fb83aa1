// Products of few rows with 4-bit weights: act(X W^T + bias) and
// act(X Wg^T) * (X Wu^T), W = (code - zero) * scale in groups of GROUP columns.
//
// A tile is 128 rows of the weights (gated: 64 of the gate, the same 64 of the other
// projection), the MMA's M, by BN rows of x, its N; its K range is divided among the
// CTAs of a cluster and joined as in ff_common.cuh.  A stage of the ring is 256
// columns: 128 bytes of each weight row, the rows of x, and the scales (and zero
// points) of its groups, all fetched by TMA, which fills what lies past N, M or K with
// zeros.
//
//   warps 0-7  a row of the weights a thread, half of a block's 128 columns: codes ->
//              code - zero in 16 bits, exact, and to TMEM (tcgen05.st), where the MMA
//              takes its A operand: the expanded weights never pass through shared
//              memory, which would bound the kernel.  Then the sums of the block before
//              from TMEM, times the scale of their group, into fp32 registers: each
//              group has sums of its own, so that no weight is rounded
//   warp 8     TMA producer
//   warp 9     tcgen05.mma, A from TMEM (two buffers), B (x) from shared memory
//
// Bound by warps 0-7: 16 x 28672 x 8192 takes 52.9 us, 31 instructions for a word of 8 codes,
// which an SM with two tiles issues at 77 % of its slots (ALU 74 %), 21 codes a clock; the SMs
// with one tile (72 of 148: 224 tiles) are half as busy.  DRAM 26 %.
#include <atomic>

#include "ff_common.cuh"

namespace ttc {
namespace ff {
namespace {

constexpr int kWarps = 8;  // of the codes
constexpr int kThreads = 32 * (kWarps + 2);
constexpr int kStageK = 256;                 // columns of a stage
constexpr int kBlockK = 128;                 // of a block: what is in a TMEM buffer
constexpr int kBlocks = kStageK / kBlockK;   // of a stage
constexpr int kWBytes = kPartCols * kStageK / 2;
constexpr int kHalfRows = 64;                // rows of a weight box
constexpr int kACols = kBlockK / 2;          // TMEM columns of a block's weights

template <int BN, int GROUP>
struct Cfg {
  static constexpr int kGroups = kStageK / GROUP;   // of a stage
  static constexpr int kSums = kBlockK / GROUP;     // of a block: accumulators of BN columns
  static constexpr int kXBox = BN * 128;            // 64 columns of x
  static constexpr int kXBytes = BN * kStageK * 2;
  static constexpr int kSBytes = kGroups * kPartCols * 2;
  static constexpr int kZBytes = kGroups * kPartCols;
  static constexpr int kStageBytes = kWBytes + kXBytes + kSBytes + kZBytes;
  static constexpr int kPartBytes = BN * kPartCols * 4;
  // two CTAs an SM where their TMEM columns fit
  static constexpr int kPerSm = kSums * BN <= 64 ? 2 : 1;
  static constexpr int kFit = (228 * 1024 / kPerSm - 1024 - 1024 - 256) / kStageBytes;
  static constexpr int kStages = kFit > 8 ? 8 : kFit;
  static constexpr int kRing = kStages * kStageBytes;
  static constexpr int kBars = 2 * kStages + 10;
  static constexpr int kSmemBytes = 1024 + kRing + kBars * 8 + 16;
  // TMEM: two buffers of weights, then two sets of sums (one where two do not fit)
  static constexpr int kTmemCols = 512 / kPerSm;
  static constexpr int kSets = 2 * kACols + 2 * kSums * BN <= kTmemCols ? 2 : 1;
  static constexpr int kSumBase = 2 * kACols;
  static_assert(kSumBase + kSets * kSums * BN <= kTmemCols, "TMEM columns");
  static_assert(kPerSm * (kSmemBytes + 1024) <= 228 * 1024, "shared memory of an SM");
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
  uint32_t idesc;
  int* status;
  uint64_t timeout_ns;
};

struct Maps {  // of the two halves of a tile's weights
  CUtensorMap W[2], S[2], Z[2], X;
};

// Codes to 16-bit operands, exact.
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

// D[tmem] (+)= A[tmem] B; b: low descriptor word (mx_umma.cuh).
__device__ __forceinline__ void tmem_mma(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\tmov.b64 db, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "r"(mx::kDescHigh)
      : "memory");
}

// Registers -> TMEM: 32 columns of this thread's lane, written when it returns.
__device__ __forceinline__ void tmem_store_32x32b_x32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};\n\t"
      "tcgen05.wait::st.sync.aligned;" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]),
      "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
      "r"(r[30]), "r"(r[31]), "r"(taddr)
      : "memory");
}

// TMEM -> registers, 8 columns (with its wait in the statement, as in sm100.cuh).
__device__ __forceinline__ void tmem_load_32x32b_x8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_load_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_load(uint32_t taddr, uint32_t (&r)[8]) {
  tmem_load_32x32b_x8(taddr, r);
}
__device__ __forceinline__ void tmem_load(uint32_t taddr, uint32_t (&r)[16]) {
  tmem_load_32x32b_x16(taddr, r);
}
__device__ __forceinline__ void tmem_load(uint32_t taddr, uint32_t (&r)[32]) {
  tmem_load_32x32b_x32(taddr, r);
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
__global__ void __launch_bounds__(kThreads, Cfg<BN, GROUP>::kPerSm)
    ff_w4_kernel(const __grid_constant__ Maps maps, const W4Args a) {
  using C = Cfg<BN, GROUP>;
  constexpr int kStages = C::kStages;
  constexpr int kSums = C::kSums;
  constexpr int kCols = BN / 2;  // rows of x whose sums a thread holds
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* smW = smem;                             // [stage][128 rows][128 bytes], swizzled
  uint8_t* smX = smW + kStages * kWBytes;          // [stage][4][BN rows][64 columns], swizzled
  uint8_t* smS = smX + kStages * C::kXBytes;       // [stage][half][group][64 rows]
  uint8_t* smZ = smS + kStages * C::kSBytes;       // the same, bytes
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kRing);
  uint64_t* empty = full + kStages;
  uint64_t* a_full = empty + kStages;  // [2] weights are in TMEM
  uint64_t* a_empty = a_full + 2;      // [2] and have been read
  uint64_t* d_full = a_empty + 2;      // [2] sums are in TMEM
  uint64_t* d_empty = d_full + 2;      // [2] and have been read
  uint64_t* drain = d_empty + 2;
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
      mbar_init(&empty[s], kWarps + 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&a_full[b], kWarps);
      mbar_init(&a_empty[b], 1);
      mbar_init(&d_full[b], 1);
      mbar_init(&d_empty[b], kWarps);
    }
    mbar_init(drain, 1);
    mbar_init(received, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == kWarps + 1) {
    tmem_alloc(tmem_slot, C::kTmemCols);
    tmem_relinquish_alloc_permit();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  grid_dependency_trigger();
  grid_dependency_wait();

  if (warp == kWarps) {
    // -------------------------------------------------------- TMA producer ---
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
        for (int c = 0; c < kStageK / 64; ++c)
          tma_load_2d(&maps.X, &full[stage], smX + stage * C::kXBytes + c * C::kXBox,
                      s * kStageK + c * 64, m0);
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
  } else if (warp == kWarps + 1) {
    // ---------------------------------------------------------- MMA issuer ---
    const uint32_t base = __shfl_sync(0xffffffffu, tmem, 0);
    int stage = 0;
    uint32_t phase = 0;
    int set = 0;
    uint32_t set_phase = 0, a_phase = 0;
    bool ok = true;
    for (int s = s_begin; s < s_end && ok; ++s) {
      ok = mx::mbar_wait_warp(&full[stage], phase, abort_flag, a.timeout_ns);
#pragma unroll
      for (int b = 0; b < kBlocks && ok; ++b) {  // (block b of a stage is in buffer b)
        ok = mx::mbar_wait_warp(&a_full[b], a_phase, abort_flag, a.timeout_ns) &&
             mx::mbar_wait_warp(&d_empty[set], set_phase ^ 1u, abort_flag, a.timeout_ns);
        if (!ok) break;
        tc_fence_after_sync();
        if (mx::elect_one()) {
          const uint32_t xl = mx::desc_low(smem_u32(smX + stage * C::kXBytes + 2 * b * C::kXBox));
          const uint32_t d = base + C::kSumBase + static_cast<uint32_t>(set * kSums * BN);
#pragma unroll
          for (int k = 0; k < kBlockK / 16; ++k)
            tmem_mma(d + (k * 16 / GROUP) * BN, base + b * kACols + k * 8,
                     xl + (k >> 2) * (C::kXBox >> 4) + (k & 3) * 2, a.idesc,
                     k * 16 % GROUP != 0 ? 1u : 0u);
          umma_commit(&a_empty[b]);
          if (b == kBlocks - 1) umma_commit(&empty[stage]);
          umma_commit(&d_full[set]);
        }
        __syncwarp();
        if (++set == C::kSets) {
          set = 0;
          set_phase ^= 1u;
        }
      }
      a_phase ^= 1u;
      if (++stage == kStages) {
        stage = 0;
        phase ^= 1u;
      }
    }
    if (!ok) {
      if (mx::elect_one()) {
        raise_abort(a.status, abort_flag, kStatusTimeoutBase | (kRoleMma << 4) | 1);
        umma_commit(drain);
        (void)mbar_wait(drain, 0, nullptr, a.timeout_ns);
      }
      __syncwarp();
    }
    if (splits > 1) mx::cluster_arrive_relaxed();
  } else {
    // --------------------------------------------- codes to TMEM, and sums ---
    const int q = warp & 3, half = warp >> 2;  // TMEM lanes; columns of a block, rows of x
    const int row = q * 32 + lane;             // of the tile
    const uint32_t lanes = static_cast<uint32_t>(q * 32) << 16;
    const uint32_t w_row = static_cast<uint32_t>(row * 128);
    // scales and zero points: [half][group][64 rows]
    const uint32_t s_row = static_cast<uint32_t>((row >> 6) * C::kGroups * 64 + (row & 63));
    float acc[kCols] = {};
    int set = 0;
    uint32_t set_phase = 0;
    bool ok = true;
    // sums of a block times the scales of its groups
    auto take_sums = [&](const float (&scale)[kSums]) {
      ok = mx::mbar_wait_warp(&d_full[set], set_phase, abort_flag, a.timeout_ns);
      if (!ok) return;
      tc_fence_after_sync();
#pragma unroll
      for (int i = 0; i < kSums; ++i) {
        uint32_t v[kCols];
        tmem_load(tmem + lanes + C::kSumBase +
                      static_cast<uint32_t>((set * kSums + i) * BN + half * kCols),
                  v);
#pragma unroll
        for (int c = 0; c < kCols; ++c) acc[c] = fmaf(scale[i], __uint_as_float(v[c]), acc[c]);
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&d_empty[set]);
      if (++set == C::kSets) {
        set = 0;
        set_phase ^= 1u;
      }
    };
    int stage = 0;
    uint32_t phase = 0, a_phase = 0;
    float before[kSums];  // scales of the block before
    for (int s = s_begin; s < s_end && ok; ++s) {
      ok = mx::mbar_wait_warp(&full[stage], phase, abort_flag, a.timeout_ns);
      if (!ok) break;
      const uint32_t w_at = smem_u32(smW + stage * kWBytes) + w_row;
      const uint32_t s_at = smem_u32(smS + stage * C::kSBytes) + 2 * s_row;
      const uint32_t z_at = smem_u32(smZ + stage * C::kZBytes) + s_row;
#pragma unroll
      for (int b = 0; b < kBlocks; ++b) {
        float scale[kSums];
#pragma unroll
        for (int i = 0; i < kSums; ++i) scale[i] = lds_scale<T>(s_at + (b * kSums + i) * 128);
        uint32_t p[32];
#pragma unroll
        for (int j = 0; j < 2; ++j) {  // 32 columns
          const int chunk = 2 * half + j;
          const uint4 w =
              lds128(w_at + (static_cast<uint32_t>((4 * b + chunk) ^ (row & 7)) << 4));
          uint32_t z = 8;
          if (a.zeros)
            z = lds_u8(z_at + static_cast<uint32_t>(b * kSums + chunk * 32 / GROUP) * 64);
          z = zero_pair<T>(z);
          dequantize8<T>(w.x, z, p + 16 * j);
          dequantize8<T>(w.y, z, p + 16 * j + 4);
          dequantize8<T>(w.z, z, p + 16 * j + 8);
          dequantize8<T>(w.w, z, p + 16 * j + 12);
        }
        if (b == kBlocks - 1) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&empty[stage]);
        }
        ok = mx::mbar_wait_warp(&a_empty[b], a_phase ^ 1u, abort_flag, a.timeout_ns);
        if (!ok) break;
        tc_fence_after_sync();
        tmem_store_32x32b_x32(tmem + lanes + static_cast<uint32_t>(b * kACols + half * 32), p);
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&a_full[b]);
        if (s != s_begin || b != 0) {
          take_sums(before);
          if (!ok) break;
        }
#pragma unroll
        for (int i = 0; i < kSums; ++i) before[i] = scale[i];
      }
      a_phase ^= 1u;
      if (++stage == kStages) {
        stage = 0;
        phase ^= 1u;
      }
    }
    if (ok) take_sums(before);
    if (!ok && lane == 0)
      raise_abort(a.status, abort_flag, kStatusTimeoutBase | (kRoleEpilogue << 4) | 1);
    // every load of this CTA has landed, and its MMAs and all of these warps have read
    // them: the ring is free for its part, and for what others send
    named_bar_sync(1, 32 * kWarps);
    if (splits > 1 && !pull) mx::cluster_arrive();
    float* part = reinterpret_cast<float*>(smem) + row;
#pragma unroll
    for (int c = 0; c < kCols; ++c) {
      const int m = half * kCols + c;
      if (m < rows) part[m * kPartCols] = acc[c];
    }
    __syncwarp();
    if (splits > 1 && pull) mx::cluster_arrive();  // the part is there to be read
  }
  __syncwarp();
  tc_fence_before_sync();
  join_and_finish<BN, kThreads>(a.out, smem, received, abort_flag, a.status, a.timeout_ns, rank,
                                splits, m0, n0, rows);
  if (warp == kWarps + 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// Into how many parts of at least two stages K is divided: as many as run in one wave (16 x
// 14336 x 4096 16.9 us in 2 parts, which share SMs, and 24.9 in 1; 16 x 8192 x 8192 18.2 and
// 27.5 with half the CTAs).  More than a wave is slower, although the 224 tiles of 16 x 28672 x
// 8192 leave 72 of 148 SMs with one CTA instead of two: 52.8 us, 55.6 in 2 parts, 57.0 in 3.
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
  int rc = encode_tmap_f16_2d(&maps.X, p.X, p.K, p.M, p.ldx, 64, BN);
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
  a.idesc = idesc_f16_f32(128, BN, false, false) |
            (p.dtype == MX_BF16 ? (1u << 7) | (1u << 10) : 0u);
  a.status = d.status;
  a.timeout_ns = d.timeout_ns;
  Launch l(dim3(static_cast<unsigned>(tiles * splits)), dim3(kThreads), C::kSmemBytes, p.stream);
  l.cluster(static_cast<unsigned>(splits));
  return launched(cudaLaunchKernelEx(&l.cfg, ff_w4_kernel<T, BN, GROUP>, maps, a));
}

template <class T, int GROUP>
int launch_rows(const W4Problem& p, const DeviceCtx& d) {
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
  if (w4_few_fits(p)) return launch_w4_few(p, d);
  return p.dtype == MX_F16 ? launch_group<__half>(p, d) : launch_group<__nv_bfloat16>(p, d);
}

}  // namespace ff
}  // namespace ttc
