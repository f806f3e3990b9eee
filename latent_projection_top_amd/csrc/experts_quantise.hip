// Rows and weights as 8-bit integers, the packed form of the weights, and the
// list of row tiles that the products work through.
#include "block_device.h"
#include "experts_launch.h"

namespace experts {

using block::BF16;
using block::F16;
using block::kWave;
using block::u32x4;

constexpr int kThreads = 256;

// The integers of values whose largest magnitude is `most`: q = rne(127 x / a),
// s = a / 127. The quotient is decided without a division: with x and a of at
// most 11 significant bits it is a border n + 1/2 exactly or at least 2^-19 of
// its size from one, and t below, a product corrected by its exact residual
// (fma), is within an ulp of it and equal where it is representable, as every
// border is. Values so small that 1 / a overflows, or so large that 127 x does,
// are scaled first, exactly.
struct Quantiser {
  float up, inv, a, s;
  __device__ __forceinline__ explicit Quantiser(float most) {
    const float shift = most < 0x1p-60f ? 0x1p+100f : most > 0x1p+60f ? 0x1p-100f : 1.f;
    a = most * shift;
    up = 127.f * shift;
    inv = a > 0.f ? 1.f / a : 0.f;
    s = most / 127.f;
    if (!(most < INFINITY)) {  // infinite or NaN: the whole row is NaN
      a = inv = up = 0.f;
      s = NAN;
    }
  }
  // the integer in the low byte; adding 1.5 x 2^23 rounds to nearest-even
  __device__ __forceinline__ uint32_t byte(float x) const {
    const float n = up > 0.f ? up * x : 0.f;
    const float t = n * inv;
    return __float_as_uint(fmaf(fmaf(-t, a, n), inv, t) + 12582912.f);
  }
  __device__ __forceinline__ uint32_t bytes(float x, float y, float z, float w) const {
    const uint32_t lo = __builtin_amdgcn_perm(byte(y), byte(x), 0x0c0c0400);
    const uint32_t hi = __builtin_amdgcn_perm(byte(w), byte(z), 0x0c0c0400);
    return lo | hi << 16;
  }
};

// Largest magnitude of a type's values as the bits of one of them, which are in
// order for what has no sign: infinity and NaN come last.
template <typename T>
__device__ __forceinline__ float magnitude(uint32_t bits) {
  return T::load((uint16_t)bits);
}

// The lists of short items and row tiles, by the first four waves of a block.
// An expert of more than kStreamRows rows has as few tiles of at most kTileRows
// as it can, of equal height.
__device__ __forceinline__ void make_lists(const int32_t* offsets, int experts, int rows, Item* area,
                                           int most_brief, int most_tiles) {
  __shared__ int2 part[kThreads / kWave];
  const int t = threadIdx.x, lane = t & (kWave - 1), wave = t / kWave;
  Item* brief = area + 1;
  Item* tiles = brief + most_brief;
  int briefs = 0, tile = 0;  // so far
  for (int e0 = 0; e0 < experts; e0 += kThreads) {
    const int e = e0 + t;
    int first = 0, n = 0;
    if (t < kThreads && e < experts) {
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
    if (t < kThreads && lane == kWave - 1) part[wave] = int2{rb, rm};
    __syncthreads();
    int ab = briefs + rb - b, am = tile + rm - m;
    for (int w = 0; w < kThreads / kWave; ++w) {
      ab += w < wave ? part[w].x : 0;
      am += w < wave ? part[w].y : 0;
      briefs += part[w].x;
      tile += part[w].y;
    }
    // offsets that overlap would make more than there is room for
    if (b != 0 && ab < most_brief) brief[ab] = Item{e, first, n, 0};
    uint64_t todo = __ballot(m > 0);  // a wave writes an expert's tiles together
    while (todo != 0) {
      const int l = __builtin_ctzll(todo);
      todo &= todo - 1;
      const int at = __shfl(am, l), end = min(at + __shfl(m, l), most_tiles);
      const Item it{__shfl(e, l), __shfl(first, l), __shfl(n, l), at};
      for (int i = at + lane; i < end; i += kWave) tiles[i] = it;
    }
    __syncthreads();
  }
  if (t == 0) *area = Item{min(briefs, most_brief), min(tile, most_tiles), 0, 0};
}

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

// Rows as integers, bound by HBM: Threads threads to a row, up to Groups times
// 16 values to a thread, which stay in registers from load to store. The block
// after the last row makes the lists.
template <typename T, int Threads, int Groups>
__global__ __launch_bounds__(Threads < kThreads ? kThreads : Threads)
void quantise_kernel(const uint16_t* x, int64_t ldx, int tokens, int k, int stride, int8_t* q, float* step,
                     const int32_t* offsets, int experts, int rows, Item* area, int most_brief, int most_tiles) {
  constexpr int kBlock = Threads < kThreads ? kThreads : Threads, kRowsPer = kBlock / Threads;
  __shared__ uint32_t part[kBlock / kWave];
  const int blocks = (tokens + kRowsPer - 1) / kRowsPer;
  if ((int)blockIdx.x == blocks) {
    make_lists(offsets, experts, rows, area, most_brief, most_tiles);
    return;
  }
  const int t = threadIdx.x % Threads, row = blockIdx.x * kRowsPer + threadIdx.x / Threads;
  const bool live = row < tokens;
  const uint16_t* in = x + (int64_t)(live ? row : tokens - 1) * ldx;
  u32x4 v[Groups][2];
#pragma unroll
  for (int i = 0; i < Groups; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = 16 * (t + Threads * i) + 8 * h;
      v[i][h] = u32x4{0, 0, 0, 0};
      if (c + 8 <= k) {
        v[i][h] = reinterpret_cast<const block::Any16*>(in + c)->v;
      } else if (c < k) {
#pragma unroll
        for (int e = 0; e < 7; ++e)
          if (c + e < k) v[i][h][e >> 1] |= (uint32_t)in[c + e] << (16 * (e & 1));
      }
    }
  u16x2 m = {0, 0};
#pragma unroll
  for (int i = 0; i < Groups; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, v[i][h][e] & 0x7fff7fffu));
  uint32_t most = max((uint32_t)m[0], (uint32_t)m[1]);
#pragma unroll
  for (int d = kWave / 2; d > 0; d /= 2) most = max(most, (uint32_t)__shfl_xor((int)most, d));
  if constexpr (Threads > kWave) {
    if ((threadIdx.x & (kWave - 1)) == 0) part[threadIdx.x / kWave] = most;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kBlock / kWave; ++w) most = max(most, part[w]);
  }
  const Quantiser z(magnitude<T>(most));
  if (!live) return;
  if (t == 0) step[row] = z.s;
  int8_t* out = q + (int64_t)row * stride;
#pragma unroll
  for (int i = 0; i < Groups; ++i) {
    const int c = 16 * (t + Threads * i);
    if (c >= stride) break;
    u32x4 b;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t lo = v[i][e >> 1][2 * (e & 1)], hi = v[i][e >> 1][2 * (e & 1) + 1];
      b[e] = z.bytes(T::load((uint16_t)lo), T::load((uint16_t)(lo >> 16)), T::load((uint16_t)hi),
                     T::load((uint16_t)(hi >> 16)));
    }
    *reinterpret_cast<u32x4*>(out + c) = b;
  }
}

template <typename T, int Threads, int Groups>
static hipError_t launch_rows(const uint16_t* x, int64_t ldx, int tokens, int k, int8_t* q, float* step,
                              const int32_t* offsets, int experts, int rows, Item* area, hipStream_t stream) {
  constexpr int kBlock = Threads < kThreads ? kThreads : Threads, kRowsPer = kBlock / Threads;
  const unsigned blocks = (unsigned)((tokens + kRowsPer - 1) / kRowsPer) + (offsets != nullptr ? 1 : 0);
  return launch_kernel(quantise_kernel<T, Threads, Groups>, dim3(blocks), dim3(kBlock), stream, x, ldx, tokens, k,
                       red_blocks(k) * kBlockRed, q, step, offsets, experts, rows, area,
                       (int)most_brief(rows, experts), (int)most_tiles(rows, experts));
}

// A wave to a row where there are enough of them to fill the CUs, else a block.
template <typename T>
static hipError_t launch_typed(const uint16_t* x, int64_t ldx, int tokens, int k, int8_t* q, float* step,
                               const int32_t* offsets, int experts, int rows, Item* area, hipStream_t stream) {
  if (k > 8192)
    return launch_rows<T, 1024, 8>(x, ldx, tokens, k, q, step, offsets, experts, rows, area, stream);
  if (k > 4096 || tokens < 1024)
    return launch_rows<T, 256, 2>(x, ldx, tokens, k, q, step, offsets, experts, rows, area, stream);
  return launch_rows<T, 64, 4>(x, ldx, tokens, k, q, step, offsets, experts, rows, area, stream);
}

hipError_t launch_quantise(int dtype, const void* x, int64_t ldx, int tokens, int k, int8_t* q, float* step,
                           const int32_t* offsets, int experts, int rows, void* area, hipStream_t stream) {
  const uint16_t* in = static_cast<const uint16_t*>(x);
  Item* items = static_cast<Item*>(area);
  return dtype == BLOCK_BF16
             ? launch_typed<BF16>(in, ldx, tokens, k, q, step, offsets, experts, rows, items, stream)
             : launch_typed<F16>(in, ldx, tokens, k, q, step, offsets, experts, rows, items, stream);
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
  *reinterpret_cast<u32x4*>(packed + (((e * tiles + tile) * blocks + b) * kBlockBytes + 16 * lane)) =
      u32x4{v[0], v[1], v[2], v[3]};
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
  uint32_t most = 0;
  for (int i = 0; i < k; ++i) most = max(most, w[(int64_t)i * n] & 0x7fffu);
  const Quantiser z(magnitude<T>(most));
  scale[e * n + c] = z.s;
  for (int i = 0; i < k; ++i) w8[(int64_t)i * n] = (int8_t)(z.byte(T::load(w[(int64_t)i * n])) & 0xff);
}

hipError_t launch_quantise_weights(int dtype, const void* w, int8_t* w8, float* scale, int experts, int k, int n,
                                   hipStream_t stream) {
  return launch_kernel(dtype == BLOCK_BF16 ? quantise_weights_kernel<BF16> : quantise_weights_kernel<F16>,
                       dim3((n + kThreads - 1) / kThreads, experts), dim3(kThreads), stream,
                       static_cast<const uint16_t*>(w), w8, scale, k, n);
}

}  // namespace experts
