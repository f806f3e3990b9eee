// Device-side building blocks of the 8-bit products (gfx950, wave64).
#pragma once

#include "block_device.h"
#include "experts_launch.h"

namespace experts {

using block::BF16;
using block::F16;
using block::kWave;
using block::u32x4;

// Of a grid of two dimensions, which may have more blocks than there is work for.
__device__ __forceinline__ int block_of_grid() { return (int)(blockIdx.y * gridDim.x + blockIdx.x); }

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));

// Lane (g, m) = (l / 16, l % 16) of the result holds column m of `b` (a row of
// x) and rows 4 g .. 4 g + 3 of `a` (columns of the weights).
__device__ __forceinline__ i32x4 mfma(u32x4 a, u32x4 b, i32x4 c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c, 0, 0,
                                              0);
}

template <bool Gated>
__device__ __forceinline__ int packed_tiles(const ProductArgs& p) {
  return (Gated ? 2 : 1) * ((p.n + 15) / 16);
}

__device__ __forceinline__ const uint8_t* packed_tile(const ProductArgs& p, int expert, int tiles, int tile) {
  return static_cast<const uint8_t*>(p.packed) + ((int64_t)expert * tiles + tile) * p.blocks * kBlockBytes;
}

// The row of x that row `row` of y is made of.
__device__ __forceinline__ int token_of(const ProductArgs& p, int row) {
  return p.token != nullptr ? min(max(p.token[row], 0), p.tokens - 1) : row;
}

// The rows that expert e has: its range of `offsets`, cut to `end`, the rows that
// there are before offsets[experts], behind which they are nobody's (their
// integers are not made).
struct Range {
  int first, rows;
};
__device__ __forceinline__ int end_of_rows(const int32_t* offsets, int experts, int rows) {
  return min(max(offsets[experts], 0), rows);
}
__device__ __forceinline__ Range range_of(const int32_t* offsets, int e, int end) {
  const int first = min(max(offsets[e], 0), end);
  return Range{first, max(min(max(offsets[e + 1], 0), end) - first, 0)};
}

// `count` (less than eight) consecutive 16-bit values, zeros after them. Every
// load is of a value that is there, so that they go out together: one by one
// where the row's end says so, each would be waited for (7 us a row's end).
__device__ __forceinline__ u32x4 edge8(const uint16_t* p, int count) {
  u32x4 v = {0, 0, 0, 0};
  if (count > 0) {
    uint32_t e[8];
#pragma unroll
    for (int t = 0; t < 7; ++t) e[t] = p[min(t, count - 1)];
    e[7] = 0;
#pragma unroll
    for (int t = 0; t < 8; t += 2) v[t / 2] = (t < count ? e[t] : 0) | (t + 1 < count ? e[t + 1] << 16 : 0);
  }
  return v;
}
__device__ __forceinline__ u32x4 load8(const uint16_t* p, int count) {
  return count >= 8 ? reinterpret_cast<const block::Any16*>(p)->v : edge8(p, count);
}

struct __attribute__((packed, aligned(4))) Any16of4 { u32x4 v; };  // 16 bytes at any 4-byte address

// C (4 or 8) consecutive columns of an expert's FP32 vector, or of a row of
// 16-bit values, `count` of them inside it.
template <int C>
__device__ __forceinline__ void load_scales(const float* s, float (&v)[C], int count) {
  if (count >= C) {
#pragma unroll
    for (int t = 0; t < C; t += 4) {
      const u32x4 x = reinterpret_cast<const Any16of4*>(s + t)->v;
#pragma unroll
      for (int f = 0; f < 4; ++f) v[t + f] = __uint_as_float(x[f]);
    }
  } else if (count > 0) {
#pragma unroll
    for (int t = 0; t < C; ++t) v[t] = s[min(t, count - 1)];
  }
}
template <typename T, int C>
__device__ __forceinline__ void load_values(const uint16_t* p, float (&v)[C], int count) {
  if (count >= C) {
    block::load_cols<T, C>(p, v, C);
  } else if (count > 0) {
    uint16_t e[C];
#pragma unroll
    for (int t = 0; t < C; ++t) e[t] = p[min(t, count - 1)];
#pragma unroll
    for (int t = 0; t < C; ++t) v[t] = T::load(e[t]);
  }
}

// What the columns of an output need: scales and the bias.
template <typename T, bool Gated, int C>
struct Columns {
  float scale[C] = {}, other[C] = {};  // other: the up product's scale, or the bias
  Columns() = default;
  __device__ __forceinline__ Columns(const ProductArgs& p, int expert, int col) {
    const int count = p.n - col;
    const int64_t at = (int64_t)expert * p.n + col;
    load_scales<C>(p.scale[0] + at, scale, count);
    if constexpr (Gated) {
      load_scales<C>(p.scale[1] + at, other, count);
    } else if (p.bias != nullptr) {
      load_values<T, C>(static_cast<const uint16_t*>(p.bias) + at, other, count);
    }
  }
};

// The end of a product: integer sums (for the gated product of both) of columns
// col .. col + C - 1 of row `row`. The channel's scale comes first: the row's
// may be as small or as large as FP32 goes.
template <typename T, bool Gated, int Act, int C>
__device__ __forceinline__ void finish(const ProductArgs& p, const Columns<T, Gated, C>& k, int row, int col,
                                       float step, const float (&sum)[C], const float (&up)[C],
                                       const float (&residual)[C]) {
  float v[C];
#pragma unroll
  for (int t = 0; t < C; ++t) {
    const float z = sum[t] * k.scale[t] * step;
    if constexpr (Gated)
      v[t] = block::activate<Act>(z).a * (up[t] * k.other[t] * step);
    else
      v[t] = block::activate<Act>(z + k.other[t]).a + residual[t];
  }
  block::store_cols<T, C>(static_cast<typename T::raw*>(p.y) + row * p.ldy + col, v, p.n - col);
}

template <bool Gated, typename F>
__device__ __forceinline__ void with_ending(const ProductArgs& p, F f) {
  block::with_activation(p.act, [&](auto act) __attribute__((always_inline)) {
    if constexpr (!Gated || decltype(act)::value != BLOCK_ACT_NONE) f(act);
  });
}

}  // namespace experts
