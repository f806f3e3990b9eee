// 8-bit products of few rows (up to 32 of an expert): the time is the weights'
// way from HBM.
//
// A block has one expert's rows and up to four column tiles of its packed
// weights. Its eight waves take the reduction's blocks of 64 in turn, 1 KB of a
// column tile per load, straight into the registers that the matrix cores read;
// the next blocks' loads are under way while one is multiplied. The waves'
// integer sums meet in LDS. Blocks go through the list of (expert, columns) by
// themselves, since only the device knows how long it is. Where that is too
// short to fill the CUs the reduction is also split over blocks, whose sums are
// added by the last of them to arrive: integers, so in any order the same.
#include "experts_device.h"

namespace experts {

constexpr int kWaves = 8;

// Sums between blocks of one launch: relaxed device-scope atomics, which go
// past the XCDs' L2s both ways.
__device__ __forceinline__ void put(int32_t* p, int v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ int get(const int32_t* p) {
  return __hip_atomic_load(const_cast<int32_t*>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

template <int C>
using Parts = int32_t[kWaves][kStreamRows][16 * C + 4];

// One item's columns from tile0 on, its split-th of `splits` parts of the
// reduction, with RT tiles of 16 rows.
template <typename T, bool Gated, int C, int RT>
__device__ __forceinline__ void stream_item(const ProductArgs& p, const Item& it, int tile0, int unit, int split,
                                            int splits, Parts<C>& part, uint32_t& arrived) {
  typedef typename T::raw raw;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int lane = threadIdx.x & (kWave - 1), g = lane >> 4, m = lane & 15;
  const int tiles = packed_tiles<Gated>(p);
  const int b0 = (int)((int64_t)p.blocks * split / splits) + wave;
  const int b1 = (int)((int64_t)p.blocks * (split + 1) / splits);
  const int count = b1 > b0 ? (b1 - b0 + kWaves - 1) / kWaves : 0;

  const uint8_t* w[C];
  const int8_t* q[RT];
#pragma unroll
  for (int c = 0; c < C; ++c)
    w[c] = packed_tile(p, it.expert, tiles, min(tile0 + c, tiles - 1)) + (int64_t)b0 * kBlockBytes + 16 * lane;
#pragma unroll
  for (int r = 0; r < RT; ++r)
    q[r] = p.q + ((int64_t)token_of(p, it.row + min(16 * r + m, it.rows - 1)) * p.blocks + b0) * kBlockRed + 16 * g;

  struct Step {
    u32x4 w[C], x[RT];
  };
  auto fetch = [&](Step& d, int i) __attribute__((always_inline)) {
#pragma unroll
    for (int c = 0; c < C; ++c) d.w[c] = *reinterpret_cast<const u32x4*>(w[c] + (int64_t)i * kWaves * kBlockBytes);
#pragma unroll
    for (int r = 0; r < RT; ++r) d.x[r] = *reinterpret_cast<const u32x4*>(q[r] + (int64_t)i * kWaves * kBlockRed);
  };
  i32x4 acc[C][RT] = {};
  auto multiply = [&](const Step& d) __attribute__((always_inline)) {
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int r = 0; r < RT; ++r) acc[c][r] = mfma(d.w[c], d.x[r], acc[c][r]);
  };
  if (count > 0) {
    Step d0, d1;
    fetch(d0, 0);
    int i = 0;
#pragma unroll 1
    for (; i + 2 < count; i += 2) {
      fetch(d1, i + 1);
      __builtin_amdgcn_sched_barrier(0);
      multiply(d0);
      fetch(d0, i + 2);
      __builtin_amdgcn_sched_barrier(0);
      multiply(d1);
    }
    if (i + 1 < count) {
      fetch(d1, i + 1);
      __builtin_amdgcn_sched_barrier(0);
      multiply(d0);
      multiply(d1);
    } else {
      multiply(d0);
    }
  }

  // lane (g, m) holds row 16 r + m, columns 16 c + 4 g .. + 3
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int r = 0; r < RT; ++r) *reinterpret_cast<i32x4*>(&part[wave][16 * r + m][16 * c + 4 * g]) = acc[c][r];
  __syncthreads();

  constexpr int kQuads = 4 * C;  // groups of 4 packed columns
  auto sums = [&](int row, int quad) __attribute__((always_inline)) {
    i32x4 v = {};
#pragma unroll
    for (int k = 0; k < kWaves; ++k) v += *reinterpret_cast<const i32x4*>(&part[k][row][4 * quad]);
    return v;
  };
  bool last = true;
  int32_t* units = p.partial + (int64_t)unit * splits * kUnitInts;
  if (splits > 1) {
    for (int id = threadIdx.x; id < it.rows * kQuads; id += kWave * kWaves) {
      const i32x4 v = sums(id / kQuads, id % kQuads);
#pragma unroll
      for (int t = 0; t < 4; ++t) put(units + (int64_t)split * kUnitInts + 4 * id + t, v[t]);
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // this wave's sums are out
    __syncthreads();
    if (threadIdx.x == 0) {
      uint32_t* c = p.counters + 16 * unit;
      arrived = __hip_atomic_fetch_add(c, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      if (arrived == (uint32_t)splits - 1) __hip_atomic_store(c, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    last = arrived == (uint32_t)splits - 1;
  }
  if (last) {
    constexpr int kOut = Gated ? kQuads / 2 : kQuads;  // groups of 4 output columns
    const int out0 = (Gated ? tile0 / 2 : tile0) * 16;
    with_ending<Gated>(p, [&](auto act) __attribute__((always_inline)) {
      for (int id = threadIdx.x; id < it.rows * kOut; id += kWave * kWaves) {
        const int row = id / kOut, o = id % kOut, col = out0 + 4 * o;
        if (col >= p.n) continue;
        const int quad = Gated ? o / 4 * 8 + o % 4 : o;
        i32x4 v = {}, u = {};
        if (splits > 1) {
          for (int s = 0; s < splits; ++s)
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              const int32_t* e = units + (int64_t)s * kUnitInts + 4 * (row * kQuads + quad) + t;
              v[t] += get(e);
              if constexpr (Gated) u[t] += get(e + 16);
            }
        } else {
          v = sums(row, quad);
          if constexpr (Gated) u = sums(row, quad + 4);
        }
        const int64_t r = it.row + row;
        const Columns<T, Gated, 4> k(p, it.expert, col);
        float sum[4], up[4], residual[4] = {};
        if (!Gated && p.residual != nullptr)
          block::load_cols<T, 4>(static_cast<const raw*>(p.residual) + r * p.ldr + col, residual, p.n - col);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          sum[t] = (float)v[t];
          up[t] = (float)u[t];
        }
        finish<T, Gated, decltype(act)::value, 4>(p, k, (int)r, col, p.step[token_of(p, (int)r)], sum, up, residual);
      }
    });
  }
  __syncthreads();  // before the next item's sums
}

template <typename T, bool Gated, int C>
__global__ __launch_bounds__(kWave * kWaves) __attribute__((amdgpu_waves_per_eu(4, 4)))
void stream_kernel(ProductArgs p) {
  __shared__ __attribute__((aligned(16))) Parts<C> part;
  __shared__ uint32_t arrived;
  const int groups = (packed_tiles<Gated>(p) + C - 1) / C;
  const int items = p.lists.counts != nullptr ? p.lists.counts[0] : 1;
  const int64_t total = (int64_t)items * groups;
  if (total == 0) return;
  int splits = 1;
  if (total < kSplitUnits * 3 / 4)
    splits = min(kSplitUnits / (int)total, max(p.blocks / kWaves, 1));
  for (int64_t at = blockIdx.x; at < total * splits; at += gridDim.x) {
    const int unit = (int)(at / splits), split = (int)(at % splits);  // (more than one: at < kSplitUnits)
    const int i = (int)(at / splits / groups), group = (int)(at / splits % groups);
    const Item it = p.lists.counts != nullptr ? p.lists.brief[i] : Item{0, 0, p.rows, 0};
    if (it.rows <= 16)
      stream_item<T, Gated, C, 1>(p, it, group * C, unit, split, splits, part, arrived);
    else
      stream_item<T, Gated, C, 2>(p, it, group * C, unit, split, splits, part, arrived);
  }
}

template <typename T, bool Gated>
static hipError_t launch_typed(const ProductArgs& p, int experts, hipStream_t stream) {
  const int64_t tiles = (Gated ? 2 : 1) * column_tiles(p.n);
  const int64_t items = p.lists.counts != nullptr ? most_brief(p.rows, experts) : 1;
  // two blocks to a CU
  const dim3 grid(512), block(kWave * kWaves);
  if (items * tiles <= 512 * 2) return launch_kernel(stream_kernel<T, Gated, 2>, grid, block, stream, p);
  return launch_kernel(stream_kernel<T, Gated, 4>, grid, block, stream, p);
}

hipError_t launch_stream(int dtype, const ProductArgs& p, int experts, hipStream_t stream) {
  if (dtype == BLOCK_BF16)
    return p.gated ? launch_typed<BF16, true>(p, experts, stream) : launch_typed<BF16, false>(p, experts, stream);
  return p.gated ? launch_typed<F16, true>(p, experts, stream) : launch_typed<F16, false>(p, experts, stream);
}

}  // namespace experts
