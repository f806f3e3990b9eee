// Rows taken to their choices' places and brought back (gather, combine and
// their gradients).
#include "block_device.h"
#include "experts_launch.h"

namespace experts {

using block::BF16;
using block::F16;
using block::F32;
using block::kWave;

// Eight columns of a row, `count` of them inside it.
template <typename T>
__device__ __forceinline__ void load8(const typename T::raw* p, float (&v)[8], int count) {
  if constexpr (sizeof(typename T::raw) == 2) {
    block::load_cols<T, 8>(p, v, count);
  } else {
#pragma unroll
    for (int t = 0; t < 8; ++t) v[t] = t < count ? p[t] : 0.f;
  }
}

template <typename T>
__device__ __forceinline__ void store8(typename T::raw* p, const float (&v)[8], int count) {
  if constexpr (sizeof(typename T::raw) == 2) {
    block::store_cols<T, 8>(p, v, count);
  } else {
#pragma unroll
    for (int t = 0; t < 8; ++t)
      if (t < count) p[t] = v[t];
  }
}

// A wave per choice: its row goes out and, for dweights, meets the sorted row.
template <typename T>
__global__ __launch_bounds__(kWave) void spread_kernel(RowsArgs p) {
  typedef typename T::raw raw;
  const int lane = threadIdx.x, r = blockIdx.x, j = blockIdx.y;
  const int at = p.place[(int64_t)r * p.topk + j];
  const bool on = (uint32_t)at < (uint32_t)p.capacity;
  const raw* x = static_cast<const raw*>(p.plain) + r * p.ld_plain;
  float dot = 0.f;
  if (on) {
    const float w = p.weights != nullptr && p.to_sorted != nullptr ? p.weights[(int64_t)r * p.topk + j] : 1.f;
    for (int c = 8 * lane; c < p.width; c += 8 * kWave) {
      float v[8], s[8];
      load8<T>(x + c, v, p.width - c);
      if (p.dweights != nullptr) {
        load8<T>(static_cast<const raw*>(p.sorted) + at * p.ld_sorted + c, s, p.width - c);
#pragma unroll
        for (int t = 0; t < 8; ++t) dot = fmaf(v[t], s[t], dot);
      }
      if (p.to_sorted != nullptr) {
#pragma unroll
        for (int t = 0; t < 8; ++t) v[t] *= w;
        store8<T>(static_cast<raw*>(p.to_sorted) + at * p.ld_to_sorted + c, v, p.width - c);
      }
    }
  }
  if (p.dweights == nullptr) return;
  for (int d = kWave / 2; d > 0; d /= 2) dot += __shfl_xor(dot, d);
  if (lane == 0) p.dweights[(int64_t)r * p.topk + j] = on ? dot : 0.f;
}

template <typename T>
__global__ __launch_bounds__(kWave) void collect_kernel(RowsArgs p) {
  typedef typename T::raw raw;
  const int r = blockIdx.x, c = 8 * (kWave * blockIdx.y + threadIdx.x), count = p.width - c;
  if (count <= 0) return;
  float sum[8] = {}, v[8];
  for (int j = 0; j < p.topk; ++j) {
    const int at = p.place[(int64_t)r * p.topk + j];
    if ((uint32_t)at >= (uint32_t)p.capacity) continue;
    const float w = p.weights != nullptr ? p.weights[(int64_t)r * p.topk + j] : 1.f;
    load8<T>(static_cast<const raw*>(p.sorted) + at * p.ld_sorted + c, v, count);
#pragma unroll
    for (int t = 0; t < 8; ++t) sum[t] = fmaf(w, v[t], sum[t]);
  }
  if (p.residual != nullptr) {
    load8<T>(static_cast<const raw*>(p.residual) + r * p.ld_residual + c, v, count);
#pragma unroll
    for (int t = 0; t < 8; ++t) sum[t] += v[t];
  }
  store8<T>(static_cast<raw*>(p.to_plain) + r * p.ld_to_plain + c, sum, count);
}

hipError_t launch_spread(int dtype, const RowsArgs& p, hipStream_t stream) {
  const dim3 grid(p.rows, p.topk);
  return launch_kernel(dtype == BLOCK_BF16 ? spread_kernel<BF16> : dtype == BLOCK_F16 ? spread_kernel<F16>
                                                                                      : spread_kernel<F32>,
                       grid, dim3(kWave), stream, p);
}

hipError_t launch_collect(int dtype, const RowsArgs& p, hipStream_t stream) {
  const dim3 grid(p.rows, (p.width + 8 * kWave - 1) / (8 * kWave));
  return launch_kernel(dtype == BLOCK_BF16 ? collect_kernel<BF16> : dtype == BLOCK_F16 ? collect_kernel<F16>
                                                                                       : collect_kernel<F32>,
                       grid, dim3(kWave), stream, p);
}

}  // namespace experts
