// Rows and weights as 8-bit integers, the packed form of the weights, and the
// list of row tiles that the products work through.
#include "block_device.h"
#include "experts_quantiser.h"

namespace experts {

using block::BF16;
using block::F16;
using block::kWave;
using block::u32x4;

constexpr int kThreads = 256;

// The lists of a product's items, by the first four waves of a block. An
// expert's rows are as few tiles of at most kTileRows as there can be, of equal
// height.
__device__ __forceinline__ void make_lists(const QuantiseArgs& p) {
  __shared__ int4 part[kThreads / kWave];
  const int t = threadIdx.x, lane = t & (kWave - 1), wave = t / kWave;
  Item* lists[3] = {p.area + 1, p.area + 1 + p.most_brief, p.area + 1 + p.most_brief + p.most_mid};
  const int most[3] = {p.most_brief, p.most_mid, p.most_tiles};
  const int end = end_of_rows(p.offsets, p.experts, p.rows);
  int4 done = {0, 0, 0, 0};
  for (int e0 = 0; e0 < p.experts; e0 += kThreads) {
    const int e = e0 + t;
    const auto [first, n] = t < kThreads && e < p.experts ? range_of(p.offsets, e, end) : Range{0, 0};
    // this thread's items: how many, of which list
    const int kind = p.way == kBrief ? 0 : p.way == kFew ? 1 : n > kStreamRows ? 2 : p.way == kTogether ? 1 : 0;
    const int height = kind == 0 ? kStreamRows : kind == 1 ? kMidRows : kTileRows;
    const int m = (n + height - 1) / height;
    // sums over the block, and before this thread
    int4 r = {kind == 0 ? m : 0, kind == 1 ? m : 0, kind == 2 ? m : 0, 0}, before = r, all = {0, 0, 0, 0};
    for (int d = 1; d < kWave; d *= 2) {
      const int x = __shfl_up(r.x, d), y = __shfl_up(r.y, d), z = __shfl_up(r.z, d);
      if (lane >= d) r = int4{r.x + x, r.y + y, r.z + z, 0};
    }
    if (t < kThreads && lane == kWave - 1) part[wave] = r;
    __syncthreads();
    before = int4{r.x - before.x, r.y - before.y, r.z - before.z, 0};
    for (int w = 0; w < kThreads / kWave; ++w) {
      const int4 s = part[w];
      if (w < wave) before = int4{before.x + s.x, before.y + s.y, before.z + s.z, 0};
      all = int4{all.x + s.x, all.y + s.y, all.z + s.z, 0};
    }
    __syncthreads();
    const int start = kind == 0 ? done.x + before.x : kind == 1 ? done.y + before.y : done.z + before.z;
    // offsets that overlap would make more than there is room for
    if (m == 1 && start < most[kind]) lists[kind][start] = Item{e, first, n, start};
    uint64_t todo = __ballot(m > 1);  // a wave writes an expert's tiles together
    while (todo != 0) {
      const int l = __builtin_ctzll(todo);
      todo &= todo - 1;
      const int k = __shfl(kind, l), at = __shfl(start, l), count = __shfl(m, l);
      const int high = k == 0 ? kStreamRows : kMidRows, of = __shfl(e, l), row = __shfl(first, l), rows = __shfl(n, l);
      for (int i = lane; i < count && at + i < most[k]; i += kWave)
        lists[k][at + i] = k == 2 ? Item{of, row, rows, at}
                                  : Item{of, row + i * high, min(rows - i * high, high), at};
    }
    done = int4{done.x + all.x, done.y + all.y, done.z + all.z, 0};
  }
  if (t == 0) *p.area = Item{min(done.x, most[0]), min(done.y, most[1]), min(done.z, most[2]), 0};
}

// Rows as integers, bound by HBM: Threads threads to a row, up to Groups times
// 16 values to a thread, which stay in registers from load to store. The block
// after the last row makes the lists. 4096 x 3584: 11 us, 44 MB at 4 TB/s; a few
// rows 4.6 us, the chain of load, largest magnitude, store and, by expert, lists.
template <typename T, int Threads, int Groups>
__global__ __launch_bounds__(Threads < kThreads ? kThreads : Threads) void quantise_kernel(QuantiseArgs p) {
  constexpr int kBlock = Threads < kThreads ? kThreads : Threads, kRowsPer = kBlock / Threads;
  __shared__ uint32_t part[kBlock / kWave];
  const int blocks = (p.tokens + kRowsPer - 1) / kRowsPer, k = p.k;
  const int block = block_of_grid();
  if (block >= blocks) {
    if (block == blocks && p.offsets != nullptr) make_lists(p);
    return;
  }
  // rows behind the last expert's are nobody's (65536 rows of 2048 of which an
  // eighth is kept, and their products of 512 columns: 103 us with them, 43)
  const int tokens = p.sorted ? end_of_rows(p.offsets, p.experts, p.rows) : p.tokens;
  if (block * kRowsPer >= tokens) return;
  const int t = threadIdx.x % Threads, row = block * kRowsPer + threadIdx.x / Threads;
  const bool live = row < tokens;
  const uint16_t* in = p.x + (int64_t)(live ? row : tokens - 1) * p.ldx;
  u32x4 v[Groups][2];
#pragma unroll
  for (int i = 0; i < Groups; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = 16 * (t + Threads * i) + 8 * h;
      v[i][h] = load8(in + c, k - c);
    }
  u16x2 m = {0, 0};
#pragma unroll
  for (int i = 0; i < Groups; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) m = larger(m, v[i][h]);
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
  if (t == 0) p.step[row] = z.s;
  int8_t* out = p.q + (int64_t)row * p.stride;
#pragma unroll
  for (int i = 0; i < Groups; ++i) {
    const int c = 16 * (t + Threads * i);
    if (c >= p.stride) break;
    *reinterpret_cast<u32x4*>(out + c) = z.template sixteen<T>(v[i][0], v[i][1]);
  }
}

template <typename T, int Threads, int Groups>
static hipError_t launch_rows(const QuantiseArgs& p, hipStream_t stream) {
  constexpr int kBlock = Threads < kThreads ? kThreads : Threads, kRowsPer = kBlock / Threads;
  const int64_t blocks = (p.tokens + kRowsPer - 1) / kRowsPer + (p.offsets != nullptr ? 1 : 0);
  return launch_kernel(quantise_kernel<T, Threads, Groups>, grid_of(blocks), dim3(kBlock), stream, p);
}

// A wave to a row where its registers hold one, else a block (with a product of 16
// columns behind it, 4096 x 2048: 17.0 us, as a block 17.7; 4096 x 1024: 13.0 and
// 14.6; in wider rows a wave would have twice the registers: 4096 x 3584 23.5 and
// 22.6).
template <typename T>
static hipError_t launch_typed(const QuantiseArgs& p, hipStream_t stream) {
  if (p.k > 8192) return launch_rows<T, 1024, 8>(p, stream);
  if (p.k > 2048) return launch_rows<T, 256, 2>(p, stream);
  return launch_rows<T, 64, 2>(p, stream);
}

hipError_t launch_quantise(int dtype, const QuantiseArgs& p, hipStream_t stream) {
  return dtype == BLOCK_BF16 ? launch_typed<BF16>(p, stream) : launch_typed<F16>(p, stream);
}

// ---------------------------------------------------------------- weights --

// Once per set of weights, so neither kernel is tuned. A thread writes 16 bytes of
// the packed form.
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
