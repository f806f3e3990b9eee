// Rows and weights as 8-bit integers, the packed form of the weights, and the
// list of row tiles that the products work through.
#include "block_device.h"
#include "experts_launch.h"

namespace experts {

using block::BF16;
using block::F16;
using block::kWave;

constexpr int kThreads = 256;

// The integers of values whose largest magnitude is a: q = rne(127 x / a), s =
// a / 127. The quotient is decided without a division: with x and a of at most
// 11 significant bits it is a border n + 1/2 exactly or at least 2^-19 of its
// size from one, and t below, a product corrected by its exact residual (fma),
// is within an ulp of it and equal where it is representable, as every border
// is. Values so small that 1 / a overflows, or so large that 127 x does, are
// scaled first, exactly.
struct Quantiser {
  float up, inv, a, s;
  __device__ __forceinline__ explicit Quantiser(float most) {
    up = most < 0x1p-60f ? 0x1p+100f : most > 0x1p+60f ? 0x1p-100f : 1.f;
    a = most * up;
    inv = a > 0.f ? 1.f / a : 0.f;
    s = most / 127.f;
    if (!(most < INFINITY)) {  // infinite or NaN: the whole row is NaN
      a = inv = 0.f;
      s = NAN;
    }
  }
  __device__ __forceinline__ int operator()(float x) const {
    const float n = a > 0.f ? 127.f * (x * up) : 0.f;
    float t = n * inv;
    t = fmaf(fmaf(-t, a, n), inv, t);
    return (int)__builtin_rintf(t);
  }
};

// Largest magnitude, NaN if there is one.
__device__ __forceinline__ float wider(float m, float x) {
  const float v = fabsf(x);
  return v > m || v != v ? v : m;
}

// A block per row; the block after the last row makes the list of items.
template <typename T>
__global__ __launch_bounds__(kThreads) void quantise_kernel(const uint16_t* x, int64_t ldx, int tokens, int k,
                                                            int stride, int8_t* q, float* step,
                                                            const int32_t* offsets, int experts, int rows,
                                                            Item* items, int32_t* count) {
  __shared__ float part[kThreads / kWave];
  __shared__ int scan[kThreads];
  const int t = threadIdx.x;
  if ((int)blockIdx.x == tokens) {
    int base = 0;
    for (int e0 = 0; e0 < experts; e0 += kThreads) {
      const int e = e0 + t;
      int first = 0, n = 0;
      if (e < experts) {
        first = min(max(offsets[e], 0), rows);
        n = max(min(max(offsets[e + 1], 0), rows) - first, 0);
      }
      const int tiles = (n + kItemRows - 1) / kItemRows;
      scan[t] = tiles;
      __syncthreads();
      for (int d = 1; d < kThreads; d *= 2) {
        const int v = t >= d ? scan[t - d] : 0;
        __syncthreads();
        scan[t] += v;
        __syncthreads();
      }
      const int most = rows / kItemRows + min(rows, experts);
      for (int i = 0; i < tiles; ++i) {
        const int at = base + scan[t] - tiles + i;
        if (at < most) items[at] = Item{e, first + i * kItemRows, min(n - i * kItemRows, kItemRows), 0};
      }
      base += scan[kThreads - 1];
      __syncthreads();
    }
    if (t == 0) *count = min(base, rows / kItemRows + min(rows, experts));
    return;
  }
  const uint16_t* row = x + (int64_t)blockIdx.x * ldx;
  int8_t* out = q + (int64_t)blockIdx.x * stride;
  float most = 0.f;
  for (int c = t; c < k; c += kThreads) most = wider(most, T::load(row[c]));
  for (int d = kWave / 2; d > 0; d /= 2) most = wider(most, __shfl_xor(most, d));
  if ((t & (kWave - 1)) == 0) part[t / kWave] = most;
  __syncthreads();
  most = 0.f;
  for (int w = 0; w < kThreads / kWave; ++w) most = wider(most, part[w]);
  const Quantiser z(most);
  if (t == 0) step[blockIdx.x] = z.s;
  for (int c = t; c < stride; c += kThreads) out[c] = c < k ? (int8_t)z(T::load(row[c])) : 0;
}

hipError_t launch_quantise(int dtype, const void* x, int64_t ldx, int tokens, int k, int8_t* q, float* step,
                           const int32_t* offsets, int experts, int rows, Item* items, int32_t* count,
                           hipStream_t stream) {
  const unsigned blocks = (unsigned)tokens + (offsets != nullptr ? 1 : 0);
  return launch_kernel(dtype == BLOCK_BF16 ? quantise_kernel<BF16> : quantise_kernel<F16>, dim3(blocks),
                       dim3(kThreads), stream, static_cast<const uint16_t*>(x), ldx, tokens, k,
                       red_blocks(k) * kBlockRed, q, step, offsets, experts, rows, items, count);
}

// ---------------------------------------------------------------- weights --

// Once per set of weights. A thread writes 16 bytes of the packed form.
__global__ __launch_bounds__(kThreads) void pack_kernel(const int8_t* w0, const int8_t* w1, int planes,
                                                        uint8_t* packed, int k, int n, int blocks, int tiles) {
  const int lane = threadIdx.x & (kWave - 1);
  const int b = blockIdx.x * (kThreads / kWave) + threadIdx.x / kWave, tile = blockIdx.y;
  const int64_t e = blockIdx.z;
  if (b >= blocks) return;
  const int8_t* w = (tile % planes != 0 ? w1 : w0) + e * k * n;
  const int col = tile / planes * 16 + (lane & 15), k0 = b * kBlockRed + 16 * (lane >> 4);
  uint32_t v[4] = {};
  if (col < n)
    for (int i = 0; i < 16; ++i)
      if (k0 + i < k) v[i >> 2] |= (uint32_t)(uint8_t)w[(int64_t)(k0 + i) * n + col] << (8 * (i & 3));
  *reinterpret_cast<block::u32x4*>(packed + (((e * tiles + tile) * blocks + b) * kBlockBytes + 16 * lane)) =
      block::u32x4{v[0], v[1], v[2], v[3]};
}

hipError_t launch_pack(const int8_t* const* w, int planes, void* packed, int experts, int k, int n,
                       hipStream_t stream) {
  const int blocks = red_blocks(k), tiles = planes * column_tiles(n), per = kThreads / kWave;
  return launch_kernel(pack_kernel, dim3((blocks + per - 1) / per, tiles, experts), dim3(kThreads), stream, w[0],
                       w[planes - 1], planes, static_cast<uint8_t*>(packed), k, n, blocks, tiles);
}

// A thread per channel.
template <typename T>
__global__ __launch_bounds__(kThreads) void quantise_weights_kernel(const uint16_t* w, int8_t* w8, float* scale,
                                                                    int k, int n) {
  const int c = blockIdx.x * kThreads + threadIdx.x;
  const int64_t e = blockIdx.y;
  if (c >= n) return;
  w += e * k * n + c;
  w8 += e * k * n + c;
  float most = 0.f;
  for (int i = 0; i < k; ++i) most = wider(most, T::load(w[(int64_t)i * n]));
  const Quantiser z(most);
  scale[e * n + c] = z.s;
  for (int i = 0; i < k; ++i) w8[(int64_t)i * n] = (int8_t)z(T::load(w[(int64_t)i * n]));
}

hipError_t launch_quantise_weights(int dtype, const void* w, int8_t* w8, float* scale, int experts, int k, int n,
                                   hipStream_t stream) {
  return launch_kernel(dtype == BLOCK_BF16 ? quantise_weights_kernel<BF16> : quantise_weights_kernel<F16>,
                       dim3((n + kThreads - 1) / kThreads, experts), dim3(kThreads), stream,
                       static_cast<const uint16_t*>(w), w8, scale, k, n);
}

}  // namespace experts
