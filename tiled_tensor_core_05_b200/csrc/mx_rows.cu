// The row-wise MX operators: quantisation, its reverse, and the RMS norm with
// the residual's addition and 16-bit or MX output.  All are bound by device
// memory: each element is read once and written once.
#include <type_traits>

#include "mx_common.cuh"
#include "mx_internal.h"

namespace ttc {
namespace mx {
namespace {

// ------------------------------------------------------------------- quantise ---
// One CTA per 128 x 128 tile of X: 16 threads read a row's 256 bytes, 32 rows
// at a time, all 4 loads of a thread in flight before the first is used.  A
// block's maximum is shared by 4 lanes; the tile's 512 scale bytes are
// collected in shared memory and written as one run.  8192 x 14336 fp16 to
// MXFP8: 59 us, 6.0 TB/s (94 % of a plain copy's); to MXFP4 55 us, 5.4 TB/s.
// 256 threads with 8 loads each are slower by 3 % on 14336 x 4096 and 10 % on
// 32 x 8192, 1024 threads by 15 % on large matrices.
constexpr int kQuantThreads = 512;
constexpr int kQuantRows = kQuantThreads / 16;      // rows at a time
constexpr int kQuantLoads = kTileRows / kQuantRows;  // of a thread

template <class T, int FMT>
__global__ void __launch_bounds__(kQuantThreads)
    quantize_kernel(const uint16_t* __restrict__ X, uint8_t* __restrict__ Q,
                    uint8_t* __restrict__ S, int64_t rows, int64_t cols, int64_t ldx, int64_t ldq,
                    int tiles) {
  __shared__ uint8_t scales[kTileBytes];
  const int kt = static_cast<int>(blockIdx.x % static_cast<unsigned>(tiles));
  const int64_t rt = blockIdx.x / static_cast<unsigned>(tiles);
  const int t = threadIdx.x;
  if (t < kTileBytes / 4) reinterpret_cast<uint32_t*>(scales)[t] = 0;
  const int q = t & 15;                 // which 8 columns of the tile
  const int64_t i = 16 * static_cast<int64_t>(kt) + q;
  const int64_t left = cols - 8 * i;    // elements from here to the row's end
  const int n = left < 0 ? 0 : (left > 8 ? 8 : static_cast<int>(left));
  const int64_t row0 = rt * kTileRows + (t >> 4);
  grid_dependency_trigger();
  __syncthreads();
  grid_dependency_wait();
  uint4 v[kQuantLoads];
#pragma unroll
  for (int j = 0; j < kQuantLoads; ++j) {
    const int64_t r = row0 + kQuantRows * j;
    v[j] = make_uint4(0, 0, 0, 0);
    if (r < rows && n > 0) v[j] = load8(X + r * ldx + 8 * i, n);
  }
#pragma unroll
  for (int j = 0; j < kQuantLoads; ++j) {
    const int64_t r = row0 + kQuantRows * j;
    float y[8];
    uint32_t e[2];
    unpack8<T>(v[j], y);
    const uint32_t byte = quantize8<FMT>(y, e);
    if (r < rows && n > 0) {
      store_elements<FMT>(Q + r * ldq, i, e, n);
      const int rr = (t >> 4) + kQuantRows * j;
      if ((q & 3) == 0) scales[(rr & 31) * 16 + (rr >> 5) * 4 + (q >> 2)] = static_cast<uint8_t>(byte);
    }
  }
  __syncthreads();
  if (t < kTileBytes / 16)
    reinterpret_cast<uint4*>(S + static_cast<int64_t>(blockIdx.x) * kTileBytes)[t] =
        reinterpret_cast<const uint4*>(scales)[t];
}

// ----------------------------------------------------------------- dequantise ---
// The same tile, 16 rows at a time: with 512 threads, 4 elements of 8 bytes in
// flight each are too few (14336 x 4096 MXFP4 4 % slower).  8192 x 14336 MXFP8:
// 55 us, 6.4 TB/s; MXFP4 47 us, 6.3 TB/s.
constexpr int kDequantThreads = 256;
template <class T, int FMT>
__global__ void __launch_bounds__(kDequantThreads)
    dequantize_kernel(const uint8_t* __restrict__ Q, const uint8_t* __restrict__ S,
                      uint16_t* __restrict__ X, int64_t rows, int64_t cols, int64_t ldq,
                      int64_t ldx, int tiles) {
  const int kt = static_cast<int>(blockIdx.x % static_cast<unsigned>(tiles));
  const int64_t rt = blockIdx.x / static_cast<unsigned>(tiles);
  const int t = threadIdx.x;
  const int q = t & 15;
  const int64_t i = 16 * static_cast<int64_t>(kt) + q;
  const int64_t left = cols - 8 * i;
  const int n = left < 0 ? 0 : (left > 8 ? 8 : static_cast<int>(left));
  const int64_t row0 = rt * kTileRows + (t >> 4);
  grid_dependency_trigger();
  grid_dependency_wait();
  if (n == 0) return;
  uint2 e[8];
  uint32_t byte[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int64_t r = row0 + 16 * j;
    if (r >= rows) break;
    byte[j] = S[scale_word(r, kt, tiles) + (q >> 2)];
    if constexpr (FMT == MX_FP8) {
      const uint8_t* p = Q + r * ldq + 8 * i;
      if (n == 8) {
        e[j] = *reinterpret_cast<const uint2*>(p);
      } else {
        uint64_t w = 0;
        for (int b = 0; b < n; ++b) w |= static_cast<uint64_t>(p[b]) << (8 * b);
        e[j] = make_uint2(static_cast<uint32_t>(w), static_cast<uint32_t>(w >> 32));
      }
    } else {
      const uint8_t* p = Q + r * ldq + 4 * i;
      e[j].y = 0;
      if (n >= 7) {
        e[j].x = *reinterpret_cast<const uint32_t*>(p);
      } else {
        e[j].x = 0;
        for (int b = 0; 2 * b < n; ++b) e[j].x |= static_cast<uint32_t>(p[b]) << (8 * b);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int64_t r = row0 + 16 * j;
    if (r >= rows) break;
    float f[8];
    if constexpr (FMT == MX_FP8) {
      const float2 a = from_e4m3x2(e[j].x), b = from_e4m3x2(e[j].x >> 16);
      const float2 c = from_e4m3x2(e[j].y), d = from_e4m3x2(e[j].y >> 16);
      f[0] = a.x, f[1] = a.y, f[2] = b.x, f[3] = b.y;
      f[4] = c.x, f[5] = c.y, f[6] = d.x, f[7] = d.y;
    } else {
      from_e2m1x8(e[j].x, f);
    }
    const float x = scale_value(byte[j]);
#pragma unroll
    for (int b = 0; b < 8; ++b) f[b] *= x;  // exact unless the product leaves fp32's range
    store8(X + r * ldx + 8 * i, pack8<T>(f), n);
  }
}

// ------------------------------------------------------------------- RMS norm ---
// y = h s w, s = 1 / sqrt(mean(h^2) + eps), h = X or X + R rounded to T.
//
// blockDim.x threads share a row, each with the 16-byte vectors threadIdx.x +
// v blockDim.x of it (V of them in registers; V = 0 reads h twice), so that 4
// consecutive lanes hold a block of 32.  What a thread does once for a row
// (sums across lanes and warps, the square root, addresses: some 250
// instructions) is shared by 8 V elements, so many rows take V = 4 and few
// threads each; few rows take more threads with fewer vectors, for latency.
//
// Precision: an MX element is decided by rounding at half steps, where the
// last bits of y matter.  h^2 and h w are exact in fp32 (products of two
// 16-bit values; a row of bf16 whose squares leave fp32's range is taken times
// a power of two, in a function of its own: 48.4 us a call as below in bf16,
// 49.4 with that row's registers in this one); the squares
// are summed with their rounding errors (two-sum) and then in fp64; s is held
// as two fp32 numbers.  y in fp32 is on the same side of every value halfway
// between two outputs as the exact y, unless it lies on such a value itself,
// which its low bits show; only then is it rounded to odd (truncated, the last
// bit set when anything was cut off), which the rounding that follows cannot
// tell from the exact value.  So every output is the formula's value rounded
// once, up to about 2^-43 relative, at the price of two more instructions an
// element than a plain fp32 product.
//
// 8192 x 4096 fp16 with residual to MXFP8: 45 us, 5.2 TB/s (81 % of a plain
// copy's; 40 us without any of the arithmetic, 42 with plain sums of squares).
// Rows prefetched by a persistent grid: 57 us, the registers cost more
// occupancy than the prefetch brings; 8 vectors a thread 66 us.
// With V = 0 (beyond 16384 columns, h read twice) 2048 x 32768 to MXFP8 takes 139
// us, 3.4 TB/s.
constexpr int64_t kSms = 148;  // of a B200, to choose V

struct NormArgs {
  const uint16_t *X, *R, *W;
  uint16_t* H;
  void* Y;
  uint8_t* S;
  int64_t rows, cols, ldx, ldr, ldh, ldy;
  double inv_cols;
  float eps;
};

__device__ __forceinline__ float2 sub2(float2 a, float2 b) {
  return __ffma2_rn(b, make_float2(-1.0f, -1.0f), a);
}

// acc + err += v^2, pair by pair, with the rounding error of each sum kept.
__device__ __forceinline__ void add_square(float2& acc, float2& err, float2 v) {
  const float2 q = __fmul2_rn(v, v);
  const float2 s = __fadd2_rn(acc, q);
  const float2 b = sub2(s, acc);
  err = __fadd2_rn(err, __fadd2_rn(sub2(acc, sub2(s, b)), sub2(q, b)));
  acc = s;
}

// p (sh + sl) rounded to odd in fp32.  The residual of p sh (exact, by fma)
// and p sl together can pass half a step, so they are added in and the
// remainder taken (fast two-sum) before the truncation is decided.
__device__ __forceinline__ float scale_odd(float p, float sh, float sl) {
  const float a = p * sh;
  const float r = fmaf(p, sl, fmaf(p, sh, -a));
  const float y = a + r;
  const float e = r - (y - a);
  uint32_t b = __float_as_uint(y);
  if (e != 0.0f) b = (b - ((e < 0.0f) != (y < 0.0f) ? 1u : 0u)) | 1u;
  // a zero with its sign, an infinity and NaN as they are
  return a != 0.0f && fabsf(a) < __uint_as_float(0x7F800000u) ? __uint_as_float(b) : a;
}

// 16-bit additions, each rounded once.
template <class T>
__device__ __forceinline__ uint4 add8(const uint4& a, const uint4& b);
template <>
__device__ __forceinline__ uint4 add8<__half>(const uint4& a, const uint4& b) {
  uint4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    reinterpret_cast<__half2*>(&r)[i] = __hadd2_rn(reinterpret_cast<const __half2*>(&a)[i],
                                                   reinterpret_cast<const __half2*>(&b)[i]);
  return r;
}
template <>
__device__ __forceinline__ uint4 add8<__nv_bfloat16>(const uint4& a, const uint4& b) {
  uint4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    reinterpret_cast<__nv_bfloat162*>(&r)[i] =
        __hadd2_rn(reinterpret_cast<const __nv_bfloat162*>(&a)[i],
                   reinterpret_cast<const __nv_bfloat162*>(&b)[i]);
  return r;
}

// 1 / sqrt(v): the approximate instruction (2^-22) and one Newton step in
// fp64 (2^-43); outside fp32's comfortable range, and for 0, inf and NaN, the
// division.
__device__ __forceinline__ double inverse_sqrt(double v) {
  if (!(v > 1e-30 && v < 1e30)) return 1.0 / sqrt(v);
  const double r = static_cast<double>(rsqrtf(static_cast<float>(v)));
  return r * fma(-0.5 * v * r, r, 1.5);
}

// The low bits of an fp32 value that are all 0 halfway between two values of
// the output type (and on them).
template <class T, int FMT>
constexpr uint32_t kTieMask = FMT == MX_FP8   ? 0x7FFFFu
                              : FMT == MX_FP4 ? 0x1FFFFFu
                              : std::is_same<T, __half>::value ? 0xFFFu
                                                                                 : 0x7FFFu;

template <int V>
constexpr int kNormThreads = V >= 4 ? 512 : 1024;

template <class T, int FMT>
__device__ __noinline__ void norm_row_scaled(const NormArgs& a, float c);

// The row of this thread; with kScaled, its h, which has been stored, is taken
// times c.
template <class T, int FMT, int V, bool kScaled>
__device__ __forceinline__ void norm_row(const NormArgs& a, float c) {
  __shared__ double part[32];
  const int tpr = blockDim.x;
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  const bool live = row < a.rows;
  const int cols = static_cast<int>(a.cols);
  const int whole = live ? cols >> 3 : 0;  // vectors of 8 elements; then `tail` elements
  const int tail = live ? cols & 7 : 0;
  const int tiles = static_cast<int>(scale_tiles(a.cols));
  // vectors a thread walks over: all of the row's 128-column tiles
  const int steps = V > 0 ? V : (16 * tiles + tpr - 1) / tpr;
  auto load = [&](const uint16_t* p, int i) {
    if (i < whole) return *reinterpret_cast<const uint4*>(p + 8 * static_cast<int64_t>(i));
    if (i == whole && tail != 0) return load8(p + 8 * static_cast<int64_t>(i), tail);
    return make_uint4(0, 0, 0, 0);
  };
  auto store = [&](uint16_t* p, int i, const uint4& v) {
    if (i < whole)
      *reinterpret_cast<uint4*>(p + 8 * static_cast<int64_t>(i)) = v;
    else if (i == whole && tail != 0)
      store8(p + 8 * static_cast<int64_t>(i), v, tail);
  };
  if (!kScaled) {
    grid_dependency_trigger();
    grid_dependency_wait();
  }

  const uint16_t* x = a.X + row * a.ldx;
  const uint16_t* r = a.R != nullptr ? a.R + row * a.ldr : nullptr;
  uint16_t* h = a.H != nullptr ? a.H + row * a.ldh : nullptr;
  uint4 hv[V > 0 ? V : 1];
  // few rows: the weights are on their way beside h, not after the sum
  constexpr bool kEarly = V == 1 || V == 2;
  uint4 early[kEarly ? V : 1];
  float2 acc = make_float2(0.0f, 0.0f), err = make_float2(0.0f, 0.0f);
  auto squares = [&](const uint4& v) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&v);
#pragma unroll
    for (int k = 0; k < 4; ++k) add_square(acc, err, unpack2<T>(w[k]));
  };
  // vector i of h once it has been stored, when there is no register copy
  auto again = [&](int i) {
    uint4 u;
    if (r != nullptr && h != nullptr) {
      u = load(h, i);  // written by this thread
    } else {
      u = load(x, i);
      if (r != nullptr) u = add8<T>(u, load(r, i));
    }
    if constexpr (kScaled) {
      uint32_t* w = reinterpret_cast<uint32_t*>(&u);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 f = __fmul2_rn(unpack2<T>(w[k]), splat2(c));
        w[k] = pack2<T>(f.x, f.y);
      }
    }
    return u;
  };
  if constexpr (V > 0) {
#pragma unroll
    for (int v = 0; v < V; ++v) hv[v] = load(x, threadIdx.x + v * tpr);
    if constexpr (kEarly) {
#pragma unroll
      for (int v = 0; v < V; ++v) early[v] = load(a.W, threadIdx.x + v * tpr);
    }
    if (r != nullptr) {
      uint4 rv[V];
#pragma unroll
      for (int v = 0; v < V; ++v) rv[v] = load(r, threadIdx.x + v * tpr);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        hv[v] = add8<T>(hv[v], rv[v]);
        if (h != nullptr) store(h, threadIdx.x + v * tpr, hv[v]);
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) squares(hv[v]);
  } else if constexpr (kScaled) {
    for (int v = 0; v < steps; ++v) squares(again(threadIdx.x + v * tpr));
  } else {
    for (int v = 0; v < steps; ++v) {
      const int i = threadIdx.x + v * tpr;
      uint4 u = load(x, i);
      if (r != nullptr) {
        u = add8<T>(u, load(r, i));
        if (h != nullptr) store(h, i, u);
      }
      squares(u);
    }
  }
  if constexpr (FMT != MX_NONE && !kScaled) {
    // the rows that the last scale tile has no row for are cleared: 16 bytes of
    // a tile are rows l, l + 32, l + 64 and l + 96, dealt out over the threads
    // of the rows that it has (word by word, one row to MXFP8 takes 7.8 instead
    // of 4.0 us with 8192 columns)
    const int64_t first = row & ~static_cast<int64_t>(kTileRows - 1);
    const int64_t left = a.rows - first;
    if (live && left < kTileRows) {
      const uint32_t have = static_cast<uint32_t>(left);
      const uint32_t chunks = 32u * static_cast<uint32_t>(tiles);
      for (uint32_t k = static_cast<uint32_t>(row - first) * tpr + threadIdx.x; k < chunks;
           k += have * tpr) {
        const uint32_t l = k & 31u;
        uint32_t* p = reinterpret_cast<uint32_t*>(
            a.S + scale_word(first, static_cast<int>(k >> 5), tiles) + 16 * l);
        if (l >= have) {
          *reinterpret_cast<uint4*>(p) = make_uint4(0, 0, 0, 0);
        } else {
#pragma unroll
          for (uint32_t j = 1; j < 4; ++j)
            if (l + 32 * j >= have) p[j] = 0;
        }
      }
    }
  }
  const int wpr = tpr >> 5;
  // mean of the squares + eps
  auto mean = [&](double eps) {
    // an infinite sum has no rounding error (inf - inf is not one)
    double sum = (isinf(acc.x) || isinf(acc.y))
                     ? static_cast<double>(acc.x) + static_cast<double>(acc.y)
                     : (static_cast<double>(acc.x) + static_cast<double>(acc.y)) +
                           (static_cast<double>(err.x) + static_cast<double>(err.y));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (wpr > 1) {
      double* mine = part + threadIdx.y * wpr;
      if (lane == 0) mine[threadIdx.x >> 5] = sum;
      __syncthreads();
      if (wpr <= 4) {
        sum = 0.0;
        for (int w = 0; w < wpr; ++w) sum += mine[w];
      } else {  // one after the other, 32 of them take 1500 cycles
        sum = lane < wpr ? mine[lane] : 0.0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      }
    }
    return fma(sum, a.inv_cols, eps);
  };
  const double m = mean(static_cast<double>(a.eps) * c * c);
  // A row of bf16 whose squares leave fp32's range is read once more and taken
  // times a power of two: 2^80 takes the smallest value to 2^-53, 2^-80 the
  // largest to 2^48.  The same for all threads of the row.
  if constexpr (std::is_same<T, __nv_bfloat16>::value && !kScaled) {
    if (!(m > 0x1p-80 && m < 0x1p127)) {
      norm_row_scaled<T, FMT>(a, m < 1.0 ? 0x1p80f : 0x1p-80f);
      return;
    }
  }
  const double s = inverse_sqrt(m);
  const float sh = static_cast<float>(s);
  const float sl = static_cast<float>(s - static_cast<double>(sh));

  auto emit = [&](int i, const uint4& u, const uint4& wv) {
    const uint32_t* hw = reinterpret_cast<const uint32_t*>(&u);
    const uint32_t* ww = reinterpret_cast<const uint32_t*>(&wv);
    float f[8];
    float2 p[4];
    uint32_t low = ~0u;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      p[k] = __fmul2_rn(unpack2<T>(hw[k]), unpack2<T>(ww[k]));
      const float2 y = __ffma2_rn(p[k], splat2(sh), __fmul2_rn(p[k], splat2(sl)));
      low = min(low, min(__float_as_uint(y.x) & kTieMask<T, FMT>,
                         __float_as_uint(y.y) & kTieMask<T, FMT>));
      f[2 * k] = y.x;
      f[2 * k + 1] = y.y;
    }
    if (low == 0u) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        f[2 * k] = scale_odd(p[k].x, sh, sl);
        f[2 * k + 1] = scale_odd(p[k].y, sh, sl);
      }
    }
    if constexpr (FMT == MX_NONE) {
      store(static_cast<uint16_t*>(a.Y) + row * a.ldy, i, pack8<T>(f));
    } else {
      if (i >= whole) {  // past the row's end: 0 whatever s is
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (i > whole || k >= tail) f[k] = 0.0f;
      }
      uint32_t q[2];
      uint32_t word = quantize8<FMT>(f, q) << (8 * ((lane >> 2) & 3));
      const int n = i < whole ? 8 : (i == whole ? tail : 0);
      if (n > 0) store_elements<FMT>(static_cast<uint8_t*>(a.Y) + row * a.ldy, i, q, n);
      // the 4 blocks of a 128-column tile are 16 lanes: their bytes make a word
      word |= __shfl_xor_sync(0xffffffffu, word, 4);
      word |= __shfl_xor_sync(0xffffffffu, word, 8);
      if ((lane & 15) == 0 && live && (i >> 4) < tiles)
        *reinterpret_cast<uint32_t*>(a.S + scale_word(row, i >> 4, tiles)) = word;
    }
  };
  if constexpr (V > 0) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int i = threadIdx.x + v * tpr;
      if constexpr (kEarly)
        emit(i, hv[v], early[v]);
      else
        emit(i, hv[v], load(a.W, i));
    }
  } else {
    for (int v = 0; v < steps; ++v) {
      const int i = threadIdx.x + v * tpr;
      emit(i, again(i), load(a.W, i));
    }
  }
}

template <class T, int FMT>
__device__ __noinline__ void norm_row_scaled(const NormArgs& a, float c) {
  norm_row<T, FMT, 0, true>(a, c);
}

template <class T, int FMT, int V>
__global__ void __launch_bounds__(kNormThreads<V>)
    rms_norm_kernel(const __grid_constant__ NormArgs a) {
  norm_row<T, FMT, V, false>(a, 1.0f);
}

template <class T, int FMT, int V>
cudaError_t launch_norm(const NormProblem& p, const NormArgs& a, int threads) {
  // rows of one warp go several to a CTA
  const int64_t per_cta = threads == 32 ? (p.rows < 4 ? p.rows : 4) : 1;
  Launch l(dim3(static_cast<unsigned>((p.rows + per_cta - 1) / per_cta)),
           dim3(static_cast<unsigned>(threads), static_cast<unsigned>(per_cta)), 0, p.stream);
  return cudaLaunchKernelEx(&l.cfg, rms_norm_kernel<T, FMT, V>, a);
}

template <class T, int FMT>
int run_norm(const NormProblem& p) {
  const NormArgs a{static_cast<const uint16_t*>(p.X), static_cast<const uint16_t*>(p.R),
                   static_cast<const uint16_t*>(p.W), static_cast<uint16_t*>(p.H), p.Y,
                   static_cast<uint8_t*>(p.S), p.rows, p.cols, p.ldx, p.ldr, p.ldh, p.ldy,
                   1.0 / static_cast<double>(p.cols), p.eps};
  // vectors of a row, in whole scale tiles; V as large as leaves 1024 threads
  // an SM, and at least what the largest CTA needs
  const int64_t vecs = 16 * scale_tiles(p.cols);
  const auto threads = [&](int v) { return (vecs + 32 * v - 1) / (32 * v) * 32; };
  int v = 4;
  while (v > 1 && p.rows * threads(v) < 1024 * kSms && threads(v / 2) <= (v / 2 >= 4 ? 512 : 1024))
    v /= 2;
  const int64_t t = threads(v);
  cudaError_t e;
  if (t > (v >= 4 ? 512 : 1024))  // beyond 16384 columns
    e = launch_norm<T, FMT, 0>(p, a, 1024);
  else if (v == 4)
    e = launch_norm<T, FMT, 4>(p, a, static_cast<int>(t));
  else if (v == 2)
    e = launch_norm<T, FMT, 2>(p, a, static_cast<int>(t));
  else
    e = launch_norm<T, FMT, 1>(p, a, static_cast<int>(t));
  return launched(e);
}

template <class T, int FMT>
int run_convert(const ConvertProblem& p, bool to_mx) {
  const int64_t tiles = scale_tiles(p.cols);
  const int64_t grid = tiles * ((p.rows + kTileRows - 1) / kTileRows);
  if (grid > INT32_MAX) return GEMM_ERR_INVALID_ARG;
  Launch l(dim3(static_cast<unsigned>(grid)), dim3(to_mx ? kQuantThreads : kDequantThreads), 0,
           p.stream);
  uint16_t* x = static_cast<uint16_t*>(const_cast<void*>(p.X));
  uint8_t* q = static_cast<uint8_t*>(const_cast<void*>(p.Q));
  uint8_t* s = static_cast<uint8_t*>(const_cast<void*>(p.S));
  const cudaError_t e =
      to_mx ? cudaLaunchKernelEx(&l.cfg, quantize_kernel<T, FMT>,
                                 static_cast<const uint16_t*>(x), q, s, p.rows, p.cols, p.ldx,
                                 p.ldq, static_cast<int>(tiles))
            : cudaLaunchKernelEx(&l.cfg, dequantize_kernel<T, FMT>,
                                 static_cast<const uint8_t*>(q), static_cast<const uint8_t*>(s),
                                 x, p.rows, p.cols, p.ldq, p.ldx, static_cast<int>(tiles));
  return launched(e);
}

template <class T>
int convert_format(const ConvertProblem& p, bool to_mx) {
  return p.format == MX_FP8 ? run_convert<T, MX_FP8>(p, to_mx) : run_convert<T, MX_FP4>(p, to_mx);
}

template <class T>
int norm_format(const NormProblem& p) {
  switch (p.format) {
    case MX_FP8: return run_norm<T, MX_FP8>(p);
    case MX_FP4: return run_norm<T, MX_FP4>(p);
    default: return run_norm<T, MX_NONE>(p);
  }
}

}  // namespace

int launch_quantize(const ConvertProblem& p) {
  return p.dtype == MX_F16 ? convert_format<__half>(p, true)
                           : convert_format<__nv_bfloat16>(p, true);
}

int launch_dequantize(const ConvertProblem& p) {
  return p.dtype == MX_F16 ? convert_format<__half>(p, false)
                           : convert_format<__nv_bfloat16>(p, false);
}

int launch_rms_norm(const NormProblem& p) {
  return p.dtype == MX_F16 ? norm_format<__half>(p) : norm_format<__nv_bfloat16>(p);
}

}  // namespace mx
}  // namespace ttc
