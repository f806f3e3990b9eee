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

// The lists of short items and row tiles, by one block. An expert of more than
// kStreamRows rows has as few tiles of at most kTileRows as it can, of equal
// height.
__device__ void make_lists(const int32_t* offsets, int experts, int rows, Item* area, int most_brief,
                           int most_tiles) {
  __shared__ uint2 part[kThreads / kWave];
  const int t = threadIdx.x, lane = t & (kWave - 1), wave = t / kWave;
  Item* brief = area + 1;
  Item* tiles = brief + most_brief;
  int briefs = 0, tile = 0;  // so far
  for (int e0 = 0; e0 < experts; e0 += kThreads) {
    const int e = e0 + t;
    int first = 0, n = 0;
    if (e < experts) {
      first = min(max(offsets[e], 0), rows);
      n = max(min(max(offsets[e + 1], 0), rows) - first, 0);
    }
    const int b = n > 0 && n <= kStreamRows ? 1 : 0;
    const int m = n > kStreamRows ? (n + kTileRows - 1) / kTileRows : 0;
    int rb = b, rm = m;
    for (int d = 1; d < kWave; d *= 2) {
      const int vb = __shfl_up(rb, d), vm = __shfl_up(rm, d);
      rb += lane >= d ? vb : 0;
      rm += lane >= d ? vm : 0;
    }
    if (lane == kWave - 1) part[wave] = uint2{(uint32_t)rb, (uint32_t)rm};
    __syncthreads();
    int ab = briefs + rb - b, am = tile + rm - m;
    for (int w = 0; w < kThreads / kWave; ++w) {
      ab += w < wave ? (int)part[w].x : 0;
      am += w < wave ? (int)part[w].y : 0;
      briefs += (int)part[w].x;
      tile += (int)part[w].y;
    }
    // offsets that overlap would make more than there is room for
    if (b != 0 && ab < most_brief) brief[ab] = Item{e, first, n, 0};
    for (int i = 0; i < m && am + i < most_tiles; ++i) tiles[am + i] = Item{e, first, n, am};
    __syncthreads();
  }
  if (t == 0) *area = Item{min(briefs, most_brief), min(tile, most_tiles), 0, 0};
}

// A block per row; the block after the last row makes the lists.
template <typename T>
__global__ __launch_bounds__(kThreads) void quantise_kernel(const uint16_t* x, int64_t ldx, int tokens, int k,
                                                            int stride, int8_t* q, float* step,
                                                            const int32_t* offsets, int experts, int rows, Item* area,
                                                            int most_brief, int most_tiles) {
  __shared__ float part[kThreads / kWave];
  const int t = threadIdx.x;
  if ((int)blockIdx.x == tokens) {
    make_lists(offsets, experts, rows, area, most_brief, most_tiles);
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
                           const int32_t* offsets, int experts, int rows, void* area, hipStream_t stream) {
  const unsigned blocks = (unsigned)tokens + (offsets != nullptr ? 1 : 0);
  return launch_kernel(dtype == BLOCK_BF16 ? quantise_kernel<BF16> : quantise_kernel<F16>, dim3(blocks),
                       dim3(kThreads), stream, static_cast<const uint16_t*>(x), ldx, tokens, k,
                       red_blocks(k) * kBlockRed, q, step, offsets, experts, rows, static_cast<Item*>(area),
                       (int)most_brief(rows, experts), (int)most_tiles(rows, experts));
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
