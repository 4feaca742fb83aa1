// Helpers of the tile kernels: tile order, the abort path's wait and launch
// set-up, which gemm_tile.cu shares with the CTA-pair kernels of the
// microscaled products (mx_gemm_pair.cu, mx_gemm_pair_split.cu), and the
// epilogue's bias loads and staged stores of fp16 elements, which only
// gemm_tile.cu uses.
#pragma once

#include <atomic>

#include "internal.h"
#include "sm100.cuh"

namespace ttc {

constexpr int kEpiRows = 32;    // rows per epilogue warp
constexpr int kEpiCols = 64;    // columns per epilogue chunk (128 bytes of fp16)
constexpr int kEpiBuf = kEpiRows * kEpiCols * 2;

// Grouped-panel rasterisation: consecutive tile indices sweep group_m
// tile-rows of one panel column by column, so the CTAs that run at the same
// time share A rows and B columns in L2.  Odd panels sweep their columns in
// reverse (a snake), so the first tiles of a panel reuse the B columns the
// previous panel read last.  A negative group_m gives panels of -group_m
// tile-columns swept row by row instead (the same with the roles of A and B
// exchanged).
__device__ __forceinline__ void tile_coords(int tile, int num_m, int num_n, int group_m,
                                            int& mb, int& nb) {
  if (group_m > 0) {
    const int per_group = group_m * num_n;
    const int g = tile / per_group;
    const int first_m = g * group_m;
    const int rows = min(num_m - first_m, group_m);
    const int r = tile - g * per_group;
    mb = first_m + r % rows;
    nb = r / rows;
    if (g & 1) nb = num_n - 1 - nb;
  } else {
    const int group_n = -group_m;
    const int per_group = group_n * num_m;
    const int g = tile / per_group;
    const int first_n = g * group_n;
    const int cols = min(num_n - first_n, group_n);
    const int r = tile - g * per_group;
    nb = first_n + r % cols;
    mb = r / cols;
    if (g & 1) mb = num_m - 1 - mb;
  }
}

// The 64 bias values of the chunk at column col0 as 32 packed pairs (0 past
// N): eight 16-byte loads (the same address in every lane) when the chunk
// lies inside N, else pair by pair.
__device__ __forceinline__ void load_bias_chunk(const __half* __restrict__ bias, int col0, int N,
                                                uint32_t (&bb)[32]) {
  if (col0 + kEpiCols <= N) {
    const uint4* src = reinterpret_cast<const uint4*>(bias + col0);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint4 q = __ldg(src + i);
      bb[4 * i] = q.x;
      bb[4 * i + 1] = q.y;
      bb[4 * i + 2] = q.z;
      bb[4 * i + 3] = q.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const int col = col0 + 2 * i;
      if (col + 1 < N) {
        bb[i] = __ldg(reinterpret_cast<const unsigned int*>(bias + col));
      } else {
        const unsigned short lo =
            col < N ? __ldg(reinterpret_cast<const unsigned short*>(bias + col)) : 0;
        bb[i] = lo;
      }
    }
  }
}

// The converted chunk `h` (row `lane` of a 32 x 64 fp16 box) -> 128-byte
// swizzled staging row per thread -> TMA store of the box (BOXES boxes per
// warp in turn).  Columns at and beyond N rounded down to 8 (the TMA store
// writes whole 16-byte groups) are written with plain stores.
template <int BOXES>
__device__ __forceinline__ void stage_chunk(const uint32_t* h, uint8_t* bufs, uint32_t& chunk_no,
                                            const CUtensorMap* tmC, __half* C, int64_t ldc,
                                            int M, int N, int n8, int row0, int col0, int lane) {
  uint8_t* buf = bufs + (chunk_no % BOXES) * kEpiBuf;
  // the store that last used `buf` has read it
  if (lane == 0) bulk_wait_group_read<BOXES - 1>();
  __syncwarp();
  // row `lane`, 128 bytes = 8 chunks of 16 bytes, chunk j stored at j ^ (row & 7)
  const uint32_t row_addr = smem_u32(buf) + lane * 128;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    st_shared_v4(row_addr + ((j ^ (lane & 7)) << 4), h[4 * j], h[4 * j + 1], h[4 * j + 2],
                 h[4 * j + 3]);
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    // C is written once and not read again here: evict-first keeps the
    // operand tiles that later tiles re-read in L2 (0.1-0.7 % faster)
    if (row0 < M && col0 < n8) tma_store_2d_hint(tmC, buf, col0, row0, l2_policy_evict_first());
    bulk_commit_group();
  }
  if (n8 < N && col0 + kEpiCols > n8 && col0 < N && row0 + lane < M) {
    // ragged tail columns [max(n8, col0), min(N, col0 + 64)) of this row,
    // read back from this thread's own (swizzled) staging row
    const int j_end = min(N, col0 + kEpiCols);
    __half* crow = C + static_cast<int64_t>(row0 + lane) * ldc;
    for (int j = max(n8, col0); j < j_end; ++j) {
      const int cc = j - col0;
      const uint32_t addr = row_addr + ((((cc >> 3) ^ (lane & 7)) << 4) | ((cc & 7) << 1));
      unsigned short bits;
      asm volatile("ld.shared.u16 %0, [%1];" : "=h"(bits) : "r"(addr) : "memory");
      crow[j] = __ushort_as_half(bits);
    }
  }
  ++chunk_no;
}

// Busy-wait for about `ns` nanoseconds (bounded, used on the abort path only).
__device__ __forceinline__ void spin_ns(uint64_t ns) {
  const uint64_t t0 = globaltimer_ns();
  while (globaltimer_ns() - t0 < ns) {
  }
}

// Sets the dynamic shared-memory limit of a kernel once per device.
inline bool ensure_smem_attr(const void* func, int bytes, int device, std::atomic<uint64_t>& done) {
  const uint64_t bit = 1ull << (device & 63);
  if (done.load(std::memory_order_acquire) & bit) return true;
  if (cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) !=
      cudaSuccess)
    return false;
  done.fetch_or(bit, std::memory_order_acq_rel);
  return true;
}

// Raster panel of the tile kernels in tiles: `group` > 0 rows of A per row
// panel -> that many tile-rows (at least 1); `group` < 0 columns of B per
// column panel -> minus that many tile-columns.
inline int group_tiles(int group, int tile_rows, int tile_cols) {
  if (group < 0) {
    const int g = -group / tile_cols;
    return g > 0 ? -g : -1;
  }
  const int g = group / tile_rows;
  return g > 0 ? g : 1;
}

}  // namespace ttc
