// Rows taken to their choices' places and brought back (gather, combine and
// their gradients). Bound by HBM: rows are read and written once, topk rows in
// sorted order for each token, 512 columns of a row to a wave, eight of a lane.
//
// A wave reads its token's places once, one to a lane, and takes the live ones
// from there in order, eight at a time, so that eight rows' loads are in flight
// together and a dropped choice costs nothing. (Not in the wave that holds a row's
// end inside a vector: it waits for each row's last values in turn.) Sums are
// FP32 in the order of the choices. 16-bit sorted rows pass by the caches (a
// training step of 4096 x 16 x 3584 BF16 in a graph: 460 us, else 530).
//
// That step's calls, traced one by one: gather 103 us (4.9 TB/s; a copy reaches
// 5.2), combine 88 (5.7), its backward pass 204 (4.8), gather's like combine. 8 x 16 x
// 7168: combine 4.4 us, a launch and three trips one after the other: places and
// weights, the residual, rows. A wave is a block of its own where rows are
// only read together (8 x 16 x 7168 with a row to a block 6.1 us, larger ones the
// same); where a row's products are summed over its columns, a row is a block's.
#include "experts_device.h"

namespace experts {

using block::F32;

constexpr int kLaneCols = 8, kWaveCols = kLaneCols * kWave;
constexpr int kGroup = 8;  // rows in flight

// Eight columns of a row as they are in memory.
template <typename T>
struct Cols {
  static constexpr int kWords = 2 * (int)sizeof(typename T::raw);
  uint32_t w[kWords];

  // `count` of them inside the row. Once: the row is not read again (rows in
  // sorted order, which together are larger than the caches), written likewise.
  template <bool Once = false>
  __device__ __forceinline__ void load(const typename T::raw* p, int count) {
    auto get = [](const u32x4* q) { return Once ? __builtin_nontemporal_load(q) : *q; };
    if constexpr (sizeof(typename T::raw) == 2) {
      if (count >= 8) {
        const u32x4 x = get(&reinterpret_cast<const block::Any16*>(p)->v);
#pragma unroll
        for (int t = 0; t < 4; ++t) w[t] = x[t];
      } else {
        const u32x4 x = edge8(p, count);
#pragma unroll
        for (int t = 0; t < 4; ++t) w[t] = x[t];
      }
    } else if (count >= 8) {
      const u32x4 x = get(&reinterpret_cast<const Any16of4*>(p)->v);
      const u32x4 y = get(&reinterpret_cast<const Any16of4*>(p + 4)->v);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        w[t] = x[t];
        w[4 + t] = y[t];
      }
    } else {
#pragma unroll
      for (int t = 0; t < 8; ++t) w[t] = __float_as_uint(p[min(t, count - 1)]);
#pragma unroll
      for (int t = 0; t < 8; ++t) w[t] = t < count ? w[t] : 0;
    }
  }
  template <bool Once = false>
  __device__ __forceinline__ void store(typename T::raw* p, int count) const {
    auto put = [](u32x4* q, u32x4 v) {
      if (Once)
        __builtin_nontemporal_store(v, q);
      else
        *q = v;
    };
    if constexpr (sizeof(typename T::raw) == 2) {
      if (count >= 8) {
        put(&reinterpret_cast<block::Any16*>(p)->v, u32x4{w[0], w[1], w[2], w[3]});
      } else {
#pragma unroll
        for (int t = 0; t < 7; ++t)
          if (t < count) p[t] = (uint16_t)(w[t >> 1] >> (16 * (t & 1)));
      }
    } else if (count >= 8) {
      put(&reinterpret_cast<Any16of4*>(p)->v, u32x4{w[0], w[1], w[2], w[3]});
      put(&reinterpret_cast<Any16of4*>(p + 4)->v, u32x4{w[4], w[5], w[6], w[7]});
    } else {
#pragma unroll
      for (int t = 0; t < 8; ++t)
        if (t < count) p[t] = __uint_as_float(w[t]);
    }
  }
  __device__ __forceinline__ float get(int t) const {
    if constexpr (sizeof(typename T::raw) == 2)
      return T::load((uint16_t)(w[t >> 1] >> (16 * (t & 1))));
    else
      return __uint_as_float(w[t]);
  }
  __device__ __forceinline__ void set(const float (&v)[8]) {
    if constexpr (sizeof(typename T::raw) == 2) {
#pragma unroll
      for (int t = 0; t < 4; ++t) w[t] = T::store2(v[2 * t], v[2 * t + 1]);
    } else {
#pragma unroll
      for (int t = 0; t < 8; ++t) w[t] = __float_as_uint(v[t]);
    }
  }
};

// A token's choices, one to a lane.
struct Choices {
  int place;
  float weight;
  uint64_t live;
  __device__ __forceinline__ Choices(const RowsArgs& p, int r, const float* weights) {
    const int lane = threadIdx.x & (kWave - 1);
    const int64_t at = (int64_t)r * p.topk + lane;
    place = lane < p.topk ? p.place[at] : -1;
    weight = weights != nullptr && lane < p.topk ? weights[at] : 1.f;
    live = __ballot((uint32_t)place < (uint32_t)p.capacity);
  }
  // the next kGroup live ones, the last of them repeated; returns how many
  __device__ __forceinline__ int next(int (&at)[kGroup], float (&w)[kGroup], int (&which)[kGroup]) {
    // (a scalar of its own: compared in 64 bits, 8 x 16 x 7168 takes 4.1 us instead of 4.0)
    const int n = __builtin_amdgcn_readfirstlane(min((int)__popcll(live), kGroup));
    int j = 0;
#pragma unroll
    for (int q = 0; q < kGroup; ++q) {
      if (live != 0) j = __builtin_ctzll(live);
      live &= live - 1;
      at[q] = __builtin_amdgcn_readlane(place, j);
      w[q] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(weight), j));
      which[q] = j;
    }
    return n;
  }
};

__device__ __forceinline__ int wave_of_grid() {
  return __builtin_amdgcn_readfirstlane(block_of_grid() * (int)(blockDim.x / kWave) + (int)threadIdx.x / kWave);
}

// Whether rows in sorted order pass by the caches where they are only read or only
// written. FP32 rows do not: a lane's eight columns are two accesses there, each
// of a half of every 32 bytes, which past the caches meet memory apart (4096 x 16 x
// 3584: gather 434 us and 204 through them, combine 206 and 190; BF16 gather 92).
// In the backward pass, which reads and writes them, they do (411 us, else 418 to
// 435).
template <typename T>
constexpr bool kPass = sizeof(typename T::raw) == 2;

// to_sorted = plain at every place.
template <typename T>
__global__ __launch_bounds__(256) void gather_kernel(RowsArgs p, int chunks) {
  typedef typename T::raw raw;
  const int id = wave_of_grid(), r = id / chunks;
  if (r >= p.rows) return;
  const int c = (id - r * chunks) * kWaveCols + kLaneCols * (threadIdx.x & (kWave - 1));
  Cols<T> v;
  if (c < p.width) v.load(static_cast<const raw*>(p.plain) + r * p.ld_plain + c, p.width - c);
  Choices k(p, r, nullptr);
  while (k.live != 0) {
    const int j = __builtin_ctzll(k.live);
    k.live &= k.live - 1;
    const int64_t at = __builtin_amdgcn_readlane(k.place, j);
    if (c < p.width)
      v.template store<kPass<T>>(static_cast<raw*>(p.to_sorted) + at * p.ld_to_sorted + c, p.width - c);
  }
}

// to_plain = the weighted sum of sorted rows, and the residual.
template <typename T>
__global__ __launch_bounds__(kWave) void collect_kernel(RowsArgs p, int chunks) {
  typedef typename T::raw raw;
  const int id = wave_of_grid(), r = id / chunks;
  if (r >= p.rows) return;
  const int c = (id - r * chunks) * kWaveCols + kLaneCols * (threadIdx.x & (kWave - 1)), count = p.width - c;
  const bool inside = count > 0;  // lanes past the row's end stay: places and weights are read out of them
  Choices k(p, r, p.weights);
  Cols<T> res;
  if (inside && p.residual != nullptr) res.load(static_cast<const raw*>(p.residual) + r * p.ld_residual + c, count);
  float sum[8] = {};
  while (k.live != 0) {
    int at[kGroup], which[kGroup];
    float w[kGroup];
    Cols<T> v[kGroup];
    const int n = k.next(at, w, which);
    if (inside) {
#pragma unroll
      for (int q = 0; q < kGroup; ++q)
        v[q].template load<kPass<T>>(static_cast<const raw*>(p.sorted) + at[q] * p.ld_sorted + c, count);
#pragma unroll
      for (int q = 0; q < kGroup; ++q)
        if (q < n)
#pragma unroll
          for (int t = 0; t < 8; ++t) sum[t] = fmaf(w[q], v[q].get(t), sum[t]);
    }
  }
  if (!inside) return;
  if (p.residual != nullptr)
#pragma unroll
    for (int t = 0; t < 8; ++t) sum[t] += res.get(t);
  res.set(sum);
  res.store(static_cast<raw*>(p.to_plain) + r * p.ld_to_plain + c, count);
}

// Eight sums over a wave's lanes at once: each step halves the lanes and the
// sums that a lane has, so that ten exchanges do what 48 would. Sum q ends in
// lanes 8 q .. 8 q + 7 and is returned by lane q.
__device__ __forceinline__ float reduce8(const float (&v)[8]) {
  const int lane = threadIdx.x & (kWave - 1);
  float a[4], b[2], s;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const float keep = lane & 32 ? v[q + 4] : v[q], give = lane & 32 ? v[q] : v[q + 4];
    a[q] = keep + __shfl_xor(give, 32);
  }
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const float keep = lane & 16 ? a[q + 2] : a[q], give = lane & 16 ? a[q] : a[q + 2];
    b[q] = keep + __shfl_xor(give, 16);
  }
  {
    const float keep = lane & 8 ? b[1] : b[0], give = lane & 8 ? b[0] : b[1];
    s = keep + __shfl_xor(give, 8);
  }
  s += __shfl_xor(s, 4);
  s += __shfl_xor(s, 2);
  s += __shfl_xor(s, 1);
  return __shfl(s, 8 * (lane & 7));
}

// A block per token, 512 columns of the row to a wave at a time: to_sorted =
// weight * plain, and the products of plain and sorted rows.
template <typename T>
__global__ __launch_bounds__(1024) void backward_kernel(RowsArgs p) {
  typedef typename T::raw raw;
  __shared__ float part[1024 / kWave][EXPERTS_MAX_TOPK];
  const int r = blockIdx.x, lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), waves = blockDim.x / kWave;
  const bool dots = p.dweights != nullptr;
  const raw* x = static_cast<const raw*>(p.plain) + r * p.ld_plain;
  Choices k(p, r, p.to_sorted != nullptr ? p.weights : nullptr);
  const uint64_t all = k.live;
  Cols<T> v;
  const int first = wave * kWaveCols + kLaneCols * lane;
  const bool one = waves * kWaveCols >= p.width;  // a row is one pass
  if (one && first < p.width) v.load(x + first, p.width - first);
  while (k.live != 0) {
    int at[kGroup], which[kGroup];
    float w[kGroup], dot[kGroup] = {};
    const int n = k.next(at, w, which);
#pragma unroll 1
    for (int c = first; c < p.width; c += waves * kWaveCols) {
      const int count = p.width - c;
      Cols<T> s[kGroup];
      if (dots)
#pragma unroll
        for (int q = 0; q < kGroup; ++q)
          s[q].template load<true>(static_cast<const raw*>(p.sorted) + at[q] * p.ld_sorted + c, count);
      if (!one) v.load(x + c, count);
      if (p.to_sorted != nullptr)
#pragma unroll
        for (int q = 0; q < kGroup; ++q)
          if (q < n) {
            float y[8];
            Cols<T> out;
#pragma unroll
            for (int t = 0; t < 8; ++t) y[t] = w[q] * v.get(t);
            out.set(y);
            out.template store<true>(static_cast<raw*>(p.to_sorted) + at[q] * p.ld_to_sorted + c, count);
          }
      if (dots)
#pragma unroll
        for (int q = 0; q < kGroup; ++q)
#pragma unroll
          for (int t = 0; t < 8; ++t) dot[q] = fmaf(v.get(t), s[q].get(t), dot[q]);
    }
    if (dots) {
      const float s = reduce8(dot);
      int j = which[0];
#pragma unroll
      for (int q = 1; q < kGroup; ++q) j = lane == q ? which[q] : j;
      if (lane < n) part[wave][j] = s;
    }
  }
  if (!dots) return;
  __syncthreads();
  if (wave == 0 && lane < p.topk) {
    float s = 0.f;
    if (all >> lane & 1)
      for (int i = 0; i < waves; ++i) s += part[i][lane];
    p.dweights[(int64_t)r * p.topk + lane] = s;
  }
}

hipError_t launch_spread(int dtype, const RowsArgs& p, hipStream_t stream) {
  const int chunks = (p.width + kWaveCols - 1) / kWaveCols;
  if (p.weights == nullptr && p.dweights == nullptr) {
    const dim3 grid = grid_of(((int64_t)p.rows * chunks + 3) / 4);
    return launch_kernel(dtype == BLOCK_BF16 ? gather_kernel<BF16> : dtype == BLOCK_F16 ? gather_kernel<F16>
                                                                                        : gather_kernel<F32>,
                         grid, dim3(256), stream, p, chunks);
  }
  return launch_kernel(dtype == BLOCK_BF16 ? backward_kernel<BF16> : dtype == BLOCK_F16 ? backward_kernel<F16>
                                                                                        : backward_kernel<F32>,
                       dim3(p.rows), dim3(kWave * (chunks < 16 ? chunks : 16)), stream, p);
}

hipError_t launch_collect(int dtype, const RowsArgs& p, hipStream_t stream) {
  const int chunks = (p.width + kWaveCols - 1) / kWaveCols;
  const dim3 grid = grid_of((int64_t)p.rows * chunks);
  return launch_kernel(dtype == BLOCK_BF16 ? collect_kernel<BF16> : dtype == BLOCK_F16 ? collect_kernel<F16>
                                                                                       : collect_kernel<F32>,
                       grid, dim3(kWave), stream, p, chunks);
}

}  // namespace experts
