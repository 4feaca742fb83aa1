// Elementwise kernels of the feed-forward operators: the gradients of the two
// projections, and the bias fill of products over no elements.
#include "ff_common.cuh"

namespace ttc {
namespace ff {
namespace {

constexpr int kThreads = 256;

// dG = dH U act'(G), dU = dH act(G): 8 columns a thread, 16 bytes of each 16-bit
// matrix and 32 of each fp32 one.  Bound by memory: 14 bytes an element.
template <class T, int ACT>
__global__ void __launch_bounds__(kThreads)
    slope_kernel(const SlopeProblem p, int64_t vectors, int64_t total) {
  grid_dependency_trigger();
  grid_dependency_wait();
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * kThreads) {
    const int64_t row = i / vectors, col = (i - row * vectors) * 8;
    const int n = static_cast<int>(p.cols - col < 8 ? p.cols - col : 8);
    const float* g = p.G + row * p.ldg + col;
    const float* u = p.U + row * p.ldu + col;
    float gv[8], uv[8], dh[8], dg[8], du[8];
    const uint4 raw = mx::load8(static_cast<const uint16_t*>(p.dH) + row * p.lddh + col, n);
    if (n == 8) {
#pragma unroll
      for (int j = 0; j < 8; j += 4) {
        *reinterpret_cast<float4*>(gv + j) = __ldcs(reinterpret_cast<const float4*>(g + j));
        *reinterpret_cast<float4*>(uv + j) = __ldcs(reinterpret_cast<const float4*>(u + j));
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        gv[j] = j < n ? g[j] : 0.0f;
        uv[j] = j < n ? u[j] : 0.0f;
      }
    }
    mx::unpack8<T>(raw, dh);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float value, slope;
      value_and_slope<ACT>(gv[j], value, slope);
      dg[j] = dh[j] * uv[j] * slope;
      du[j] = dh[j] * value;
    }
    mx::store8(static_cast<uint16_t*>(p.dG) + row * p.lddg + col, mx::pack8<T>(dg), n);
    mx::store8(static_cast<uint16_t*>(p.dU) + row * p.lddu + col, mx::pack8<T>(du), n);
  }
}

template <class T>
__global__ void __launch_bounds__(kThreads)
    fill_kernel(const uint16_t* bias, uint16_t* Y, int64_t rows, int64_t cols, int64_t ldy,
                int act) {
  grid_dependency_trigger();
  grid_dependency_wait();
  const int64_t total = rows * cols;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * kThreads) {
    const int64_t r = i / cols, c = i - r * cols;
    const float b = bias != nullptr ? mx::unpack2<T>(bias[c]).x : 0.0f;
    with_act(act, [&](auto k) {
      const float2 y = ff_activate2<decltype(k)::value>(make_float2(b, b));
      Y[r * ldy + c] = static_cast<uint16_t>(mx::pack2<T>(y.x, y.y));
    });
  }
}

unsigned blocks_for(int64_t items, int sm_count) {
  const int64_t blocks = (items + kThreads - 1) / kThreads, most = 16ll * sm_count;
  return static_cast<unsigned>(blocks < most ? blocks : most);
}

template <class T>
int launch_slope_typed(const SlopeProblem& p, const DeviceCtx& d) {
  const int64_t vectors = (p.cols + 7) / 8, total = p.rows * vectors;
  Launch l(dim3(blocks_for(total, d.sm_count)), dim3(kThreads), 0, p.stream);
  auto go = [&](auto kern) { return launched(cudaLaunchKernelEx(&l.cfg, kern, p, vectors, total)); };
  switch (p.act) {
    case kActSilu: return go(slope_kernel<T, kActSilu>);
    case kActGelu: return go(slope_kernel<T, kActGelu>);
    case kActRelu: return go(slope_kernel<T, kActRelu>);
    default: return go(slope_kernel<T, kActNone>);
  }
}

}  // namespace

int launch_slope(const SlopeProblem& p, const DeviceCtx& d) {
  return p.dtype == MX_F16 ? launch_slope_typed<__half>(p, d)
                           : launch_slope_typed<__nv_bfloat16>(p, d);
}

int launch_bias_fill(const void* bias, void* Y, int64_t rows, int64_t cols, int64_t ldy, int dtype,
                     int act, cudaStream_t stream) {
  const int64_t blocks = (rows * cols + kThreads - 1) / kThreads;
  Launch l(dim3(static_cast<unsigned>(blocks < 4096 ? blocks : 4096)), dim3(kThreads), 0, stream);
  auto go = [&](auto kern) {
    return launched(cudaLaunchKernelEx(&l.cfg, kern, static_cast<const uint16_t*>(bias),
                                       static_cast<uint16_t*>(Y), rows, cols, ldy, act));
  };
  return dtype == MX_F16 ? go(fill_kernel<__half>) : go(fill_kernel<__nv_bfloat16>);
}

}  // namespace ff
}  // namespace ttc
