// Products of 8-bit rows and packed 8-bit weights, by expert.
#include "block_device.h"
#include "experts_launch.h"

namespace experts {

using block::BF16;
using block::F16;
using block::kWave;
using block::u32x4;

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ i32x4 mfma(u32x4 a, u32x4 b, i32x4 c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c, 0, 0,
                                              0);
}

// A wave per 16 rows of an item and 64 output columns, operands straight from
// memory.
template <typename T, bool Gated>
__global__ __launch_bounds__(256) void product_kernel(ProductArgs p, int experts) {
  typedef typename T::raw raw;
  constexpr int kTiles = Gated ? 8 : 4;
  const int wave = threadIdx.x / kWave, lane = threadIdx.x & (kWave - 1), g = lane >> 4, m = lane & 15;
  Item it;
  if (p.items != nullptr) {
    if ((int)blockIdx.x >= *p.count) return;
    it = p.items[blockIdx.x];
  } else {
    it = Item{0, (int)blockIdx.x * kItemRows, min(p.rows - (int)blockIdx.x * kItemRows, kItemRows), 0};
  }
  if (16 * wave >= it.rows) return;
  const bool in = 16 * wave + m < it.rows;
  const int row = it.row + min(16 * wave + m, it.rows - 1);
  const int t = p.token != nullptr ? min(max(p.token[row], 0), p.tokens - 1) : row;
  const int tiles = (Gated ? 2 : 1) * ((p.n + 15) / 16), tile0 = blockIdx.y * kTiles;
  const int8_t* q = p.q + (int64_t)t * p.blocks * kBlockRed + 16 * g;
  const uint8_t* w[kTiles];
#pragma unroll
  for (int c = 0; c < kTiles; ++c)
    w[c] = static_cast<const uint8_t*>(p.packed) +
           ((int64_t)it.expert * tiles + min(tile0 + c, tiles - 1)) * p.blocks * kBlockBytes + 16 * lane;
  i32x4 acc[kTiles] = {};
  for (int b = 0; b < p.blocks; ++b) {
    const u32x4 a = *reinterpret_cast<const u32x4*>(q + (int64_t)b * kBlockRed);
#pragma unroll
    for (int c = 0; c < kTiles; ++c)
      acc[c] = mfma(*reinterpret_cast<const u32x4*>(w[c] + (int64_t)b * kBlockBytes), a, acc[c]);
  }
  if (!in) return;
  const float step = p.step[t];
  block::with_activation(p.act, [&](auto act) __attribute__((always_inline)) {
#pragma unroll
    for (int c = 0; c < (Gated ? kTiles / 2 : kTiles); ++c) {
      const int col = blockIdx.y * 64 + 16 * c + 4 * g, count = p.n - col;
      if (count <= 0) continue;
      float v[4], bias[4] = {}, residual[4] = {};
      const int64_t at = (int64_t)it.expert * p.n + col;
      if (!Gated && p.bias != nullptr) block::load_cols<T, 4>(static_cast<const raw*>(p.bias) + at, bias, count);
      if (!Gated && p.residual != nullptr)
        block::load_cols<T, 4>(static_cast<const raw*>(p.residual) + row * p.ldr + col, residual, count);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i >= count) continue;
        if constexpr (Gated) {
          const float z = (float)acc[2 * c][i] * p.scale[0][at + i] * step;
          v[i] = block::activate<decltype(act)::value>(z).a * ((float)acc[2 * c + 1][i] * p.scale[1][at + i] * step);
        } else {
          const float z = (float)acc[c][i] * p.scale[0][at + i] * step + bias[i];
          v[i] = block::activate<decltype(act)::value>(z).a + residual[i];
        }
      }
      block::store_cols<T, 4>(static_cast<raw*>(p.y) + row * p.ldy + col, v, count);
    }
  });
}

hipError_t launch_product(int dtype, const ProductArgs& p, int experts, hipStream_t stream) {
  const int64_t items = p.items != nullptr ? most_items(p.rows, experts) : (p.rows + kItemRows - 1) / kItemRows;
  const dim3 grid((unsigned)items, (p.n + 63) / 64);
  if (dtype == BLOCK_BF16)
    return launch_kernel(p.gated ? product_kernel<BF16, true> : product_kernel<BF16, false>, grid, dim3(256),
                         stream, p, experts);
  return launch_kernel(p.gated ? product_kernel<F16, true> : product_kernel<F16, false>, grid, dim3(256), stream, p,
                       experts);
}

}  // namespace experts
