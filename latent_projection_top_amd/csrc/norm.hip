// Layer norm, forward and backward.
#include "block_device.h"

namespace block {

// Sum over the 256 threads of a block, returned to all of them; the order of
// the additions is fixed. red: 4 floats of LDS, free for reuse on return.
__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d, kWave);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  const float s = (red[0] + red[1]) + (red[2] + red[3]);
  __syncthreads();
  return s;
}

// One block per row; the variance is the mean of the centred squares.
template <typename T>
__global__ __launch_bounds__(256) void norm_kernel(NormArgs p) {
  __shared__ float red[4];
  const int64_t row = blockIdx.x;
  const typename T::raw* x = static_cast<const typename T::raw*>(p.x) + row * p.ldx;
  typename T::raw* y = static_cast<typename T::raw*>(p.y) + row * p.ldy;
  float s = 0.f;
  for (int i = threadIdx.x; i < p.width; i += 256) s += T::load(x[i]);
  const float mean = block_sum(s, red) / (float)p.width;
  float v = 0.f;
  for (int i = threadIdx.x; i < p.width; i += 256) {
    const float d = T::load(x[i]) - mean;
    v += d * d;
  }
  const float rstd = 1.f / sqrtf(block_sum(v, red) / (float)p.width + p.eps);
  for (int i = threadIdx.x; i < p.width; i += 256) {
    const float w = p.weight ? load_param(p.weight, i, p.param_dtype) : 1.f;
    const float b = p.bias ? load_param(p.bias, i, p.param_dtype) : 0.f;
    y[i] = T::store((T::load(x[i]) - mean) * rstd * w + b);
  }
  if (p.mean != nullptr && threadIdx.x == 0) {
    p.mean[row] = mean;
    p.rstd[row] = rstd;
  }
}

template <typename T>
__global__ __launch_bounds__(256) void norm_dx_kernel(NormArgs p) {
  __shared__ float red[4];
  const int64_t row = blockIdx.x;
  const typename T::raw* x = static_cast<const typename T::raw*>(p.x) + row * p.ldx;
  const typename T::raw* dy = static_cast<const typename T::raw*>(p.dy) + row * p.lddy;
  typename T::raw* dx = static_cast<typename T::raw*>(p.dx) + row * p.lddx;
  const float mean = p.mean[row], rstd = p.rstd[row];
  float s1 = 0.f, s2 = 0.f;
  for (int i = threadIdx.x; i < p.width; i += 256) {
    const float w = p.weight ? load_param(p.weight, i, p.param_dtype) : 1.f;
    const float g = w * T::load(dy[i]);
    s1 += g;
    s2 += g * ((T::load(x[i]) - mean) * rstd);
  }
  s1 = block_sum(s1, red) / (float)p.width;
  s2 = block_sum(s2, red) / (float)p.width;
  for (int i = threadIdx.x; i < p.width; i += 256) {
    const float w = p.weight ? load_param(p.weight, i, p.param_dtype) : 1.f;
    const float xh = (T::load(x[i]) - mean) * rstd;
    dx[i] = T::store(rstd * (w * T::load(dy[i]) - s1 - xh * s2));
  }
}

// Blocks of 64 columns, four row lanes each, joined in a fixed order.
template <typename T>
__global__ __launch_bounds__(256) void norm_dparam_kernel(NormArgs p) {
  __shared__ float rw[256], rb[256];
  const int col = blockIdx.x * 64 + (threadIdx.x & 63);
  float sw = 0.f, sb = 0.f;
  if (col < p.width) {
    for (int64_t r = threadIdx.x >> 6; r < p.rows; r += 4) {
      const float dy = T::load(static_cast<const typename T::raw*>(p.dy)[r * p.lddy + col]);
      const float x = T::load(static_cast<const typename T::raw*>(p.x)[r * p.ldx + col]);
      sb += dy;
      sw += dy * ((x - p.mean[r]) * p.rstd[r]);
    }
  }
  rw[threadIdx.x] = sw;
  rb[threadIdx.x] = sb;
  __syncthreads();
  const int t = threadIdx.x;
  if (t < 64 && col < p.width) {
    if (p.dweight) store_param(p.dweight, col, p.param_dtype, (rw[t] + rw[t + 64]) + (rw[t + 128] + rw[t + 192]));
    if (p.dbias) store_param(p.dbias, col, p.param_dtype, (rb[t] + rb[t + 64]) + (rb[t + 128] + rb[t + 192]));
  }
}

template <typename T>
static hipError_t norm_backward_typed(const NormArgs& p, hipStream_t stream) {
  if (p.dx != nullptr && p.rows > 0) {
    const hipError_t e = launch_kernel(norm_dx_kernel<T>, dim3((unsigned)p.rows), dim3(256), stream, p);
    if (e != hipSuccess) return e;
  }
  if (p.dweight == nullptr && p.dbias == nullptr) return hipSuccess;
  return launch_kernel(norm_dparam_kernel<T>, dim3((p.width + 63) / 64), dim3(256), stream, p);
}

hipError_t launch_norm(int dtype, const NormArgs& p, hipStream_t stream) {
  const dim3 grid((unsigned)p.rows);
  if (dtype == BLOCK_F32) return launch_kernel(norm_kernel<F32>, grid, dim3(256), stream, p);
  if (dtype == BLOCK_F16) return launch_kernel(norm_kernel<F16>, grid, dim3(256), stream, p);
  return launch_kernel(norm_kernel<BF16>, grid, dim3(256), stream, p);
}

hipError_t launch_norm_backward(int dtype, const NormArgs& p, hipStream_t stream) {
  if (dtype == BLOCK_F32) return norm_backward_typed<F32>(p, stream);
  if (dtype == BLOCK_F16) return norm_backward_typed<F16>(p, stream);
  return norm_backward_typed<BF16>(p, stream);
}

size_t norm_backward_bytes(int64_t, int) { return 0; }

}  // namespace block
