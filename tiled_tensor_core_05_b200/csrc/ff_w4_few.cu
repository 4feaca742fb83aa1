// Products of very few rows with 4-bit weights: act(X W^T + bias) and
// act(X Wg^T) * (X Wu^T), W = (code - zero) * scale in groups of GROUP columns.
//
// Besides reading the weights, the instructions that turn codes into operands bound such a
// product: an SM has to take 45 codes a clock to keep up with memory, and issues 4 x 32
// instructions.  So the codes are masked, not converted: a 16-bit pair with codes in its
// lowest bits is a pair of fp16 subnormals, code 2^-24, and with codes in the next four bits,
// code 2^-20.  The tensor cores multiply these exactly.  Four masks and a shift make
// the operands of 8 codes.  x is prepared for that once a CTA: each row, a group of
// columns at a time, as
//     x = e 2^-24 y,  e = 2^(floor(log2 max |x|) + 10),
// y in fp16 (a sixteenth of it for the columns whose codes lie in the upper bits): exactly,
// but for what lies below 2^-34 of the group's largest value.  Then, in fp32,
//     sum (code - zero) x = e (sum (code 2^-24) y - zero sum 2^-24 y),
// and the group's scale is applied to that: no weight is rounded.  (The scale comes last, so
// that fp32 holds the group's sum itself, not a part of 2^24 of it: bf16 results keep their bits
// down to bf16's smallest.)  Rows of x with infinities or with values of 2^116 and more, whose
// sums fp32 may not hold, are summed plainly.
//
// A CTA an SM goes through its tiles of 16 rows of the weights (gated: 8 of each); its
// warps take the tiles' blocks of 256 columns in turn, each with its own ring in shared
// memory that it alone fills (TMA) and reads, so that nothing waits for another warp
// but the end of a tile, and loads for the next tiles are on their way meanwhile.  TMA also
// fills what lies past N and K with zeros, so that the loop has no edges.
//
// mma.sync m16n8k16, weights times 8 rows of x.  The MMA's k-th column may be any column
// of the block, as long as it is the same one for the weights and x: the four threads that
// share a row take a quarter of a group's columns each, whole words of codes as they lie
// in memory, and 16 bytes of y for each.  y lies in the order that makes these reads of
// all lanes free of bank conflicts.  The MMA's row g of a half is row (g / 2 + 4 (g % 2)) of
// the weights for the same reason.  Gated, rows g and g + 8 of the MMA's 16 are the
// same row of the two weights, so that a thread holds both sums of an output.  The warps'
// sums are added in a fixed order.
//
// Measured (calls in turn on weights from memory), 128 columns a group: 1 x 14336 x 4096
// 12.1 us (2.5 TB/s), gated 19.5 us (3.1 TB/s), 1 x 28672 x 8192 28.4 us (4.3 TB/s), 8 rows
// 45 us.  The fixed part is 4 us (5 x 1000 x 1000).  In the largest products issue slots and
// memory are each half busy: what is left are the chains of masks and MMAs of four warps a
// scheduler.  With the weights brought by cp.async, whose addresses and edges cost as many
// instructions as the products, they took 16.5, 26.2 and 43.1 us.  12 warps: 12.5, 21.5, 31.1 us; 20:
// 12.6, 20.4, 28.0; 24: 13.7, 21.3, 29.1; 3 blocks on their way instead of 2: 12.2, 20.3,
// 28.9, and fewer rows fit.  16 rows with K divided among a cluster of 4, so that x fits,
// took 125 us, the kernel of more rows 53: sums of 16 warps and rows hold few tiles at a
// time, and everything waits at the end of each few.
#include <atomic>

#include "ff_common.cuh"

namespace ttc {
namespace ff {
namespace {

constexpr int kWarps = 16;
constexpr int kThreads = 32 * kWarps;
constexpr int kBlockK = 256;  // columns of a block
constexpr int kRows = 8;      // of x
constexpr int kTileRows = 16;
constexpr int kXBatch = 4;    // blocks of x that a warp asks for at a time
constexpr int kDepth = 2;  // blocks of a warp on their way

// A place of a ring: a block's codes, [half][row], 128-byte swizzled; and elsewhere
// its groups' scales and zero points, [group][row], for each half (gated) or both.
constexpr int kCodes = kTileRows * kBlockK / 2;
constexpr int kScales = 512;       // scales, then zero points
constexpr int kScaleHalf = 128;    // of the second weight
constexpr int kZeros = 256;
constexpr int kRingBytes = kWarps * kDepth * (kCodes + kScales);
constexpr int kFixedBytes = 1024 + kRingBytes + kWarps * kDepth * 8 + 16;

struct FewArgs {
  Tail out;
  const uint16_t* X;
  int64_t ldx;
  W4Weight w[2];
  int K, blocks, tiles;
  int round;  // tiles whose sums are held before they are added
  int* status;
  uint64_t timeout_ns;
};

struct FewMaps {
  CUtensorMap W[2], S[2], Z[2];
};

// Rows that e and the sums of y are held for: pairs.
__host__ __device__ __forceinline__ int row_pairs(int M) { return (M + 1) >> 1; }

// Bytes beside the warps' sums, and those of a tile: of M rows in pairs, 8 lanes each.
template <int GROUP>
int64_t base_bytes(int64_t M, int64_t K) {
  const int64_t blocks = (K + kBlockK - 1) / kBlockK;
  return kFixedBytes + M * blocks * (2 * kBlockK) +
         blocks * (kBlockK / GROUP) * row_pairs(static_cast<int>(M)) * 16;
}
__host__ __device__ __forceinline__ int part_bytes(int M) { return kWarps * row_pairs(M) * 128; }

__device__ __forceinline__ void mma16816(float2 (&d)[2], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0].x), "+f"(d[0].y), "+f"(d[1].x), "+f"(d[1].y)
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The bits of 2^116: from there on a row is summed plainly.  (A group's sum, of up to 128
// products with 15, stays below 2^11 times 2^116.)
constexpr uint32_t kPlainFrom = (127u + 116u) << 23;

// y, e and the sums of y of a row's block, 8 columns a lane.  bits: of the group's largest
// magnitude; a NaN's or an infinity's is above all others.
template <class T, int GROUP>
__device__ __forceinline__ uint4 prepare8(const uint4& raw, uint32_t& bits, float& e, float& sum) {
  float v[8];
  mx::unpack8<T>(raw, v);
  bits = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) bits = max(bits, __float_as_uint(fabsf(v[i])));
#pragma unroll
  for (int o = 1; o < GROUP / 8; o <<= 1) bits = max(bits, __shfl_xor_sync(0xffffffffu, bits, o));
  // floor(log2) + 127, at least 27 (y of smaller groups loses nothing: bf16's subnormals are
  // multiples of 2^-133, a sixteenth of y holds those of 2^-134), so that both powers are normal
  // numbers
  const uint32_t field = min(max(bits >> 23, 27u), 254u);
  const float inverse = __uint_as_float((268u - field) << 23);
  sum = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] *= inverse;
    sum += v[i];
  }
#pragma unroll
  for (int o = 1; o < GROUP / 8; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  sum *= 5.9604644775390625e-8f;  // 2^-24
  // NaN: the row's sums become NaN
  e = __uint_as_float(bits >= kPlainFrom ? 0x7FC00000u : (field + 10u) << 23);
  v[2] *= 0.0625f;
  v[3] *= 0.0625f;
  v[6] *= 0.0625f;
  v[7] *= 0.0625f;
  return mx::pack8<__half>(v);
}

// The sum of a row of x times a row of a weight, for rows that the split into e and y cannot
// hold.  x counts 2^-16, so that a group's sum is in range wherever the result is.
template <class T, int GROUP>
__device__ __noinline__ float plain_sum(const uint16_t* x, const W4Weight& w, int n, int K) {
  const uint8_t* q = static_cast<const uint8_t*>(w.Q) + n * w.ldq;
  float total = 0.0f;
  for (int k0 = 0; k0 < K; k0 += GROUP) {
    const int64_t i = k0 / GROUP;
    const float zero =
        w.Z == nullptr ? 8.0f : static_cast<float>(static_cast<const uint8_t*>(w.Z)[i * w.ldz + n]);
    float sum = 0.0f;
    for (int k = k0; k < min(k0 + GROUP, K); ++k) {
      // column 2 i of a word's 8 in bits 4 i, column 2 i + 1 in bits 4 i + 16
      const int byte = (k >> 3) * 4 + (k & 1) * 2 + ((k >> 2) & 1);
      const int code = (q[byte] >> ((k & 2) * 2)) & 15;
      sum = fmaf(static_cast<float>(code) - zero, 0x1p-16f * mx::unpack2<T>(x[k]).x, sum);
    }
    total = fmaf(sum, mx::unpack2<T>(static_cast<const uint16_t*>(w.S)[i * w.lds + n]).x, total);
  }
  return 0x1p16f * total;
}

template <class T, int GROUP, bool GATED>
__global__ void __launch_bounds__(kThreads, 1)
    ff_w4_few_kernel(const __grid_constant__ FewMaps maps, const FewArgs a) {
  constexpr int VEC = GROUP / 32;           // words of a thread and group
  constexpr int kGroups = kBlockK / GROUP;  // of a block
  extern __shared__ uint8_t smem_raw[];
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const bool zeros = a.w[0].Z != nullptr;
  const int N = a.out.N, M = a.out.M, blocks = a.blocks;
  const int pairs = row_pairs(M);
  uint8_t* smem = smem_raw + (-smem_u32(smem_raw) & 1023u);
  uint8_t* codes = smem + warp * (kDepth * kCodes);
  uint8_t* scales = smem + kWarps * kDepth * kCodes + warp * (kDepth * kScales);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kRingBytes) + warp * kDepth;
  // bits m and 8 + m: row m of x holds an infinity or what is as large as kPlainFrom, a NaN
  int* special = reinterpret_cast<int*>(smem + kRingBytes + kWarps * kDepth * 8);
  volatile int* abort_flag = special + 1;
  uint8_t* smX = smem + kRingBytes + kWarps * kDepth * 8 + 16;  // [row][block] y
  uint8_t* smE = smX + M * blocks * (2 * kBlockK);  // [group][pair of rows] e, e, sums of y
  // [tile of a round][warp][pair of rows][g]
  float4* parts = reinterpret_cast<float4*>(smE + blocks * kGroups * pairs * 16);
  const int tile_begin = static_cast<int>(static_cast<int64_t>(a.tiles) * blockIdx.x / gridDim.x);
  const int tile_end =
      static_cast<int>(static_cast<int64_t>(a.tiles) * (blockIdx.x + 1) / gridDim.x);
  constexpr int kTileN = GATED ? kTileRows / 2 : kTileRows;  // columns of Y

  grid_dependency_trigger();
  if (lane == 0) {
    for (int i = 0; i < kDepth; ++i) mbar_init(&full[i], 1);
    fence_barrier_init();
    tma_prefetch_desc(&maps.W[0]);
    tma_prefetch_desc(&maps.S[0]);
    if (GATED) {
      tma_prefetch_desc(&maps.W[1]);
      tma_prefetch_desc(&maps.S[1]);
    }
    if (zeros) tma_prefetch_desc(&maps.Z[0]);
    if (GATED && zeros) tma_prefetch_desc(&maps.Z[1]);
  }
  if (threadIdx.x == 0) {
    *special = 0;
    *abort_flag = 0;
  }
  __syncthreads();
  grid_dependency_wait();

  // x's first blocks are asked for before the weights, and y made after.  y: the pieces of 8
  // columns of a group in the order [v][t] (thread t's v-th), halves of 128 bytes exchanged
  // in odd rows.
  uint4 raw[kXBatch];
  auto load_x = [&](int i) {
#pragma unroll
    for (int j = 0; j < kXBatch; ++j, i += kWarps) {
      const int row = i / blocks, col = (i - row * blocks) * kBlockK + lane * 8;
      raw[j] = make_uint4(0, 0, 0, 0);
      if (row < M && col < a.K)
        raw[j] = mx::load8(a.X + row * a.ldx + col, min(8, a.K - col));
    }
  };
  load_x(warp);

  // The next block to be fetched.
  int f_tile = tile_begin, f_block = warp, ahead = 0;  // blocks asked for and not awaited
  auto next_tile = [&] {
    while (f_block >= blocks) {
      f_block -= blocks;
      ++f_tile;
    }
  };
  next_tile();
  const uint64_t policy = l2_policy_evict_first();
  const uint32_t bytes =
      kCodes + 2 * kTileRows * kGroups + (zeros ? (GATED ? 32 : 16) * kGroups : 0);
  auto fetch = [&](int place) {
    if (f_tile < tile_end) {
      if (lane == 0) {
        uint64_t* bar = &full[place];
        uint8_t *c = codes + place * kCodes, *s = scales + place * kScales;
        const int n = f_tile * kTileN;
        mbar_arrive_expect_tx(bar, bytes);
        tma_load_2d_hint(&maps.W[0], bar, c, f_block * (kBlockK / 2), n, policy);
        if (GATED)
          tma_load_2d_hint(&maps.W[1], bar, c + kCodes / 2, f_block * (kBlockK / 2), n, policy);
        tma_load_2d(&maps.S[0], bar, s, n, f_block * kGroups);
        if (GATED) tma_load_2d(&maps.S[1], bar, s + kScaleHalf, n, f_block * kGroups);
        // (16 of them, from a multiple of 16)
        if (zeros) tma_load_2d(&maps.Z[0], bar, s + kZeros, n & ~15, f_block * kGroups);
        if (GATED && zeros)
          tma_load_2d(&maps.Z[1], bar, s + kZeros + kScaleHalf, n & ~15, f_block * kGroups);
      }
      f_block += kWarps;
      ++ahead;
      next_tile();
    }
  };
#pragma unroll 1
  for (int d = 0; d < kDepth; ++d) fetch(d);

  auto prepare = [&](int i, const uint4& raw) {
    const int row = i / blocks, block = i - row * blocks;
    uint32_t bits;
    float e, sum;
    const uint4 y = prepare8<T, GROUP>(raw, bits, e, sum);
    const int in_group = lane % (4 * VEC);
    const int to = lane - in_group + in_group % VEC * 4 + in_group / VEC;
    reinterpret_cast<uint4*>(smX + i * (2 * kBlockK))[to ^ ((row & 1) << 2)] = y;
    if (in_group == 0) {
      float* at = reinterpret_cast<float*>(smE) +
                  ((block * kGroups + lane / (4 * VEC)) * pairs + (row >> 1)) * 4 + (row & 1);
      at[0] = e;
      at[2] = sum;
      if (bits >= kPlainFrom) atomicOr(special, (bits <= 0x7F800000u ? 1 : 256) << row);
    }
  };
  for (int i = warp; i < M * blocks; i += kXBatch * kWarps) {
    if (i != warp) load_x(i);
#pragma unroll
    for (int j = 0; j < kXBatch; ++j)
      if (i + j * kWarps < M * blocks) prepare(i + j * kWarps, raw[j]);
  }
  __syncthreads();

  const int x_row = min(g, M - 1);
  const uint8_t* x = smX + x_row * blocks * (2 * kBlockK);
  // pieces 0 .. 3 and 4 .. 7 of each 8
  const uint32_t x_off = (t ^ ((x_row & 1) << 2)) * 16;
  const uint8_t* e_at = smE + min(t, pairs - 1) * 16;  // of this thread's two columns
  const int row = (g >> 1) + (g & 1) * 4;              // of the half, in the weights
  // Adds the warps' sums of a tile and stores rows 2 t and 2 t + 1 of Y, columns n and (plain)
  // n + 8.
  auto finish = [&](int tile, const float4* part) {
    float4 s = part[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) {
      const float4 p = part[w * pairs * 8];
      s.x += p.x;
      s.y += p.y;
      s.z += p.z;
      s.w += p.w;
    }
    const int n = tile * kTileN + row, m = 2 * t;
    if (*special != 0) {
      auto again = [&](int i, int w, int col, float v) {
        return m + i < M && col < N && ((*special >> (m + i)) & 0x101) == 1
                   ? plain_sum<T, GROUP>(a.X + (m + i) * a.ldx, a.w[w], col, a.K)
                   : v;
      };
      s.x = again(0, 0, n, s.x);
      s.y = again(1, 0, n, s.y);
      s.z = again(0, GATED, GATED ? n : n + 8, s.z);
      s.w = again(1, GATED, GATED ? n : n + 8, s.w);
    }
    auto store = [&](int row, int col, float v) {
      if (row < M && col < N)
        a.out.Y[row * a.out.ldy + col] = static_cast<uint16_t>(mx::pack2<T>(v, v));
    };
    with_act(a.out.act, [&](auto act) {
      constexpr int ACT = decltype(act)::value;
      if (GATED) {
        const float2 y =
            __fmul2_rn(ff_activate2<ACT>(make_float2(s.x, s.y)), make_float2(s.z, s.w));
        store(m, n, y.x);
        store(m + 1, n, y.y);
      } else {
        float b0 = 0.0f, b1 = 0.0f;
        if (a.out.bias != nullptr) {
          if (n < N) b0 = mx::unpack2<T>(a.out.bias[n]).x;
          if (n + 8 < N) b1 = mx::unpack2<T>(a.out.bias[n + 8]).x;
        }
        const float2 y0 = ff_activate2<ACT>(make_float2(s.x + b0, s.y + b0));
        const float2 y1 = ff_activate2<ACT>(make_float2(s.z + b1, s.w + b1));
        store(m, n, y0.x);
        store(m + 1, n, y0.y);
        store(m, n + 8, y1.x);
        store(m + 1, n + 8, y1.y);
      }
    });
  };
  int place = 0, block = warp;
  uint32_t phase = 0;
  bool ok = true;
  for (int first = tile_begin; first < tile_end; first += a.round) {
    const int count = min(a.round, tile_end - first);
#pragma unroll 1
    for (int i = 0; i < count; ++i) {
      float2 acc[2] = {};
      const int z_from = GATED ? ((first + i) & 1) * 8 : 0;
#pragma unroll 1
      for (; block < blocks; block += kWarps) {
        if (ok) {
          ok = mx::mbar_wait_warp(&full[place], phase, abort_flag, a.timeout_ns);
          if (!ok) {
            if (lane == 0)
              raise_abort(a.status, abort_flag, kStatusTimeoutBase | (kRoleEpilogue << 4) | 1);
            // what has been asked for arrives before the CTA ends
            for (int p = place; ahead > 0; --ahead) {
              (void)mbar_wait(&full[p], phase ^ (p < place), nullptr, a.timeout_ns);
              p = p + 1 == kDepth ? 0 : p + 1;
            }
          }
          --ahead;
        }
        if (ok) {
          const uint8_t* from = codes + place * kCodes + row * 128;
          const uint16_t* s_at =
              reinterpret_cast<const uint16_t*>(scales + place * kScales) + row;
          const uint8_t* z_at = scales + place * kScales + kZeros + z_from + row;
          const uint8_t* xb[2] = {x + block * (2 * kBlockK) + x_off,
                                  x + block * (2 * kBlockK) + (x_off ^ 64)};
#pragma unroll
          for (int j = 0; j < kGroups; ++j) {
            uint32_t w[2][VEC];
            float scale[2], zero[2] = {8.0f, 8.0f};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              // word t VEC of the group: in piece 2 VEC j + t VEC / 4 of 16 bytes
              const uint8_t* p = from + h * (kCodes / 2) +
                                 ((j * VEC + t * VEC / 4) ^ row) * 16 + t * VEC % 4 * 4;
              if constexpr (VEC == 4)
                *reinterpret_cast<uint4*>(w[h]) = *reinterpret_cast<const uint4*>(p);
              else if constexpr (VEC == 2)
                *reinterpret_cast<uint2*>(w[h]) = *reinterpret_cast<const uint2*>(p);
              else
                w[h][0] = *reinterpret_cast<const uint32_t*>(p);
              constexpr int kStep = GATED ? 8 : 16;
              scale[h] = mx::unpack2<T>(s_at[j * kStep + h * (GATED ? kScaleHalf / 2 : 8)]).x;
              if (zeros)
                zero[h] = static_cast<float>(z_at[j * 16 + h * (GATED ? kScaleHalf : 8)]);
            }
            float2 sum[2] = {};
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
              const int c = j * VEC + v;  // of 4 pieces
              const uint4 y = *reinterpret_cast<const uint4*>(xb[c & 1] + (c & ~1) * 64);
              const uint32_t a0 = w[0][v], a1 = w[1][v], b0 = a0 >> 8, b1 = a1 >> 8;
              mma16816(sum, a0 & 0x000F000Fu, a1 & 0x000F000Fu, a0 & 0x00F000F0u,
                       a1 & 0x00F000F0u, y.x, y.y);
              mma16816(sum, b0 & 0x000F000Fu, b1 & 0x000F000Fu, b0 & 0x00F000F0u,
                       b1 & 0x00F000F0u, y.z, y.w);
            }
            const float4 e =
                *reinterpret_cast<const float4*>(e_at + (block * kGroups + j) * pairs * 16);
#pragma unroll
            for (int h = 0; h < 2; ++h)
              acc[h] = __ffma2_rn(
                  make_float2(scale[h], scale[h]),
                  __fmul2_rn(make_float2(e.x, e.y),
                             __ffma2_rn(make_float2(-zero[h], -zero[h]), make_float2(e.z, e.w),
                                        sum[h])),
                  acc[h]);
          }
          __syncwarp();
          fetch(place);
        }
        if (++place == kDepth) {
          place = 0;
          phase ^= 1u;
        }
      }
      block -= blocks;
      if (t < pairs)
        parts[((i * kWarps + warp) * pairs + t) * 8 + g] =
            make_float4(acc[0].x, acc[0].y, acc[1].x, acc[1].y);
    }
    __syncthreads();
    for (int i = warp; i < count; i += kWarps)
      if (t < pairs && *abort_flag == 0)
        finish(first + i, parts + (i * kWarps * pairs + t) * 8 + g);
    if (first + count < tile_end) __syncthreads();
  }
}

template <class T, int GROUP, bool GATED>
int launch(const W4Problem& p, const DeviceCtx& d) {
  static std::atomic<uint64_t> attr_done{0};
  const uint64_t bit = 1ull << (d.device & 63);
  if (!(attr_done.load(std::memory_order_acquire) & bit)) {
    if (cudaFuncSetAttribute(ff_w4_few_kernel<T, GROUP, GATED>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kMaxDynamicSmem) != cudaSuccess)
      return runtime_error();
    attr_done.fetch_or(bit, std::memory_order_acq_rel);
  }
  constexpr int kCols = GATED ? kTileRows / 2 : kTileRows, kGroups = kBlockK / GROUP;
  const int64_t row_bytes = (p.K + 7) / 8 * 4, groups = (p.K + GROUP - 1) / GROUP;
  FewMaps maps;
  FewArgs a{};
  for (int i = 0; i < 1 + GATED; ++i) {
    const W4Weight& w = p.w[i];
    a.w[i] = w;
    int rc = encode_tmap_u8_2d(&maps.W[i], w.Q, row_bytes, p.N, w.ldq, kCols);
    if (rc == 0) rc = encode_tmap_rows(&maps.S[i], w.S, 2, p.N, groups, w.lds, kCols, kGroups);
    if (rc == 0 && w.Z != nullptr)
      rc = encode_tmap_rows(&maps.Z[i], w.Z, 1, p.N, groups, w.ldz, 16, kGroups);
    if (rc != 0) return rc;
  }
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
  a.X = static_cast<const uint16_t*>(p.X);
  a.ldx = p.ldx;
  a.K = static_cast<int>(p.K);
  a.blocks = static_cast<int>((p.K + kBlockK - 1) / kBlockK);
  a.tiles = static_cast<int>((p.N + kCols - 1) / kCols);
  a.status = d.status;
  a.timeout_ns = d.timeout_ns;
  const int ctas = a.tiles < d.sm_count ? a.tiles : d.sm_count;
  const int part = part_bytes(a.out.M), base = static_cast<int>(base_bytes<GROUP>(p.M, p.K));
  const int fit = (kMaxDynamicSmem - base) / part, most = (a.tiles + ctas - 1) / ctas;
  a.round = fit < most ? fit : most;
  Launch l(dim3(static_cast<unsigned>(ctas)), dim3(kThreads),
           static_cast<size_t>(base + a.round * part), p.stream);
  return launched(cudaLaunchKernelEx(&l.cfg, ff_w4_few_kernel<T, GROUP, GATED>, maps, a));
}

template <class T, int GROUP>
int launch_gated(const W4Problem& p, const DeviceCtx& d) {
  return p.gated ? launch<T, GROUP, true>(p, d) : launch<T, GROUP, false>(p, d);
}

template <class T>
int launch_group(const W4Problem& p, const DeviceCtx& d) {
  switch (p.group) {
    case 32: return launch_gated<T, 32>(p, d);
    case 64: return launch_gated<T, 64>(p, d);
    default: return launch_gated<T, 128>(p, d);
  }
}

}  // namespace

// Up to 8 rows, as long as they fit into shared memory beside the rings (8 x 14336 x 4096
// 16.1 us; the kernel of more rows takes 17 for 16 of them; 1 x 14336 x 4096 12.1 and 16.4).
bool w4_few_fits(const W4Problem& p) {
  if (p.M > kRows) return false;
  const int64_t base = p.group == 32   ? base_bytes<32>(p.M, p.K)
                       : p.group == 64 ? base_bytes<64>(p.M, p.K)
                                       : base_bytes<128>(p.M, p.K);
  return base + part_bytes(static_cast<int>(p.M)) <= kMaxDynamicSmem;
}

int launch_w4_few(const W4Problem& p, const DeviceCtx& d) {
  return p.dtype == MX_F16 ? launch_group<__half>(p, d) : launch_group<__nv_bfloat16>(p, d);
}

}  // namespace ff
}  // namespace ttc
