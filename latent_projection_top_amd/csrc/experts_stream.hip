// 8-bit products of few rows (up to 32 of an expert): the time is the weights'
// way from HBM.
//
// A block has one expert's rows and four column tiles of its packed weights.
// Its eight waves take the reduction's blocks of 64 in turn, 1 KB of a column
// tile per load, straight into the registers that the matrix cores read; the
// next blocks' loads are under way while one is multiplied. The waves' integer
// sums meet in LDS. 512 blocks, two to a CU, so that one's sums meet while the
// other's weights arrive, go through the list of items by themselves, since only
// the device knows how long it is. Where that is too little to fill the CUs and
// the reduction is long, it is also split over blocks, whose sums are added by
// the last of them to arrive: integers, so in any order the same.
//
// Gated, 8 x 16 of 112 experts of 3584 x 4096: 33 us, 206 to 220 MB at 6.4 TB/s, more
// than a copy reaches. 8 x 2048 x 7168: 7.2 us for 15 MB, a launch and three trips to
// memory one after the other: scales and bias, rows and weights, the residual.
//
// For few rows of short reductions (Fused) the kernel reads the rows as they are
// and makes the integers itself: each wave those of its own blocks of the
// reduction, after the row's largest magnitude has gone around through LDS. It
// makes its own list of items as well.
#include "experts_device.h"
#include "experts_quantiser.h"

namespace experts {

constexpr int kWaves = 8, kThreads = kWave * kWaves;

// Sums between blocks of one launch: relaxed device-scope atomics, which go
// past the XCDs' L2s both ways.
__device__ __forceinline__ void put(int32_t* p, int v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ int get(const int32_t* p) {
  return __hip_atomic_load(const_cast<int32_t*>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

struct Shared {
  int32_t part[kWaves * kStreamRows * (16 * 4 + 4)];
  uint32_t most[kWaves][kFusedItem];
  uint32_t arrived;
};

// 16 values of a row, `count` of them inside it.
__device__ __forceinline__ void load16(const uint16_t* p, u32x4 (&v)[2], int count) {
  v[0] = load8(p, count);
  v[1] = load8(p + 8, count - 8);
}

// One item's columns from tile0 on, C column tiles of them, its split-th of
// `splits` parts of the reduction, with RT tiles of 16 rows.
template <typename T, bool Gated, int C, int RT, bool Fused, bool Split>
__device__ __forceinline__ void stream_part(const ProductArgs& p, const Item& it, int tile0, int unit, int split,
                                            int splits, Shared& shared) {
  constexpr int kPitch = 16 * C + 4;
  typedef int32_t Part[16 * RT][kPitch];
  Part* part = reinterpret_cast<Part*>(shared.part);
  static_assert(sizeof(Part) * kWaves <= sizeof(Shared::part), "LDS");
  // (not the same register as in the item before: what is made of it would
  // otherwise be kept from item to item, in more registers than there are)
  int tid = threadIdx.x;
  asm volatile("" : "+v"(tid));
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int lane = tid & (kWave - 1), g = lane >> 4, m = lane & 15;
  const int tiles = packed_tiles<Gated>(p);
  const int b0 = (Split ? (int)((int64_t)p.blocks * split / splits) : 0) + wave;
  const int b1 = Split ? (int)((int64_t)p.blocks * (split + 1) / splits) : p.blocks;
  const int count = b1 > b0 ? (b1 - b0 + kWaves - 1) / kWaves : 0;

  const uint8_t* w[C];  // uniform; lanes are 16 bytes apart
#pragma unroll
  for (int c = 0; c < C; ++c)
    w[c] = packed_tile(p, it.expert, tiles, min(tile0 + c, tiles - 1)) + (int64_t)b0 * kBlockBytes;
  int token[RT];
  const char* q[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    token[r] = token_of(p, it.row + min(16 * r + m, it.rows - 1));
    if constexpr (Fused)
      q[r] = reinterpret_cast<const char*>(p.x + token[r] * p.ldx + b0 * kBlockRed + 16 * g);
    else
      q[r] = reinterpret_cast<const char*>(p.q) + ((int64_t)token[r] * p.blocks + b0) * kBlockRed + 16 * g;
  }
  struct Step {
    u32x4 w[C], x[RT];
  };
  auto fetch = [&](Step& d, int i) __attribute__((always_inline)) {
    // past the caches: no other block reads them (16 x 3584 x 65536: 56 us, like
    // this 51) but those of the other items that an expert of many rows becomes
#pragma unroll
    for (int c = 0; c < C; ++c)
      d.w[c] = __builtin_nontemporal_load(
          reinterpret_cast<const u32x4*>(w[c] + (int64_t)i * kWaves * kBlockBytes + (uint32_t)(16 * lane)));
    if constexpr (!Fused)
#pragma unroll
      for (int r = 0; r < RT; ++r) d.x[r] = *reinterpret_cast<const u32x4*>(q[r] + (int64_t)i * kWaves * kBlockRed);
  };

  // A thread ends four columns of one row. What it needs for that is loaded before
  // the first operands (and there before them: these loads are conditional, and the
  // compiler waits where their branches meet), or after the last, where registers
  // are short.
  constexpr int kQuads = 4 * C, kOut = Gated ? 2 * C : 4 * C;  // groups of 4 packed and output columns
  static_assert(16 * RT * kQuads <= kThreads, "");
  int row, col, quad;
  Columns<T, Gated, 4> k;
  float step = 0.f;
  auto fetch_ends = [&]() __attribute__((always_inline)) {
    asm volatile("" : "+v"(tid));
    const int o = tid % kOut;
    row = tid / kOut;
    col = (Gated ? tile0 / 2 : tile0) * 16 + 4 * o;
    quad = Gated ? o / 4 * 8 + o % 4 : o;
    k = Columns<T, Gated, 4>(p, it.expert, col);
    if constexpr (!Fused) step = p.step[token_of(p, it.row + min(row, it.rows - 1))];
  };
  constexpr bool kRoom = C == 2;  // registers for them meanwhile
  if (kRoom) fetch_ends();

  i32x4 acc[C][RT] = {};
  auto multiply = [&](const Step& d) __attribute__((always_inline)) {
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int c = 0; c < C; ++c) acc[c][r] = mfma(d.w[c], d.x[r], acc[c][r]);
  };
  // Depth steps are on their way at once, as many as there are registers for.
  constexpr int kDepth = C == 2 ? 4 : RT == 1 ? 3 : 2;
  Step d[kDepth];
  if constexpr (Fused) {
    // The rows' loads go out before the weights', behind which they would have
    // to wait. (They are in one trip: the weights' are conditional as well, and have
    // arrived where the magnitudes begin.)
    u32x4 v[kFusedSteps][2];
#pragma unroll
    for (int i = 0; i < kFusedSteps; ++i)
      load16(reinterpret_cast<const uint16_t*>(q[0]) + i * kWaves * kBlockRed, v[i],
             p.k - (wave + i * kWaves) * kBlockRed - 16 * g);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int s = 0; s < kDepth; ++s)
      if (s < count) fetch(d[s], s);
    __builtin_amdgcn_sched_barrier(0);
    // the rows' largest magnitudes: of this wave's blocks, then of all
    u16x2 most = {0, 0};
#pragma unroll
    for (int i = 0; i < kFusedSteps; ++i) most = larger(larger(most, v[i][0]), v[i][1]);
    uint32_t a = max((uint32_t)most[0], (uint32_t)most[1]);
    a = max(a, (uint32_t)__shfl_xor((int)a, 16));
    a = max(a, (uint32_t)__shfl_xor((int)a, 32));
    if (g == 0) shared.most[wave][m] = a;
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");  // LDS only
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
    a = 0;
#pragma unroll
    for (int k = 0; k < kWaves; ++k) a = max(a, shared.most[k][m]);
    const Quantiser z(magnitude<T>(a));
#pragma unroll
    for (int i = 0; i < kFusedSteps; ++i)
      if (i < count) {
        d[i % kDepth].x[0] = z.template sixteen<T>(v[i][0], v[i][1]);
        multiply(d[i % kDepth]);
        __builtin_amdgcn_sched_barrier(0);
        if (i + kDepth < count) fetch(d[i % kDepth], i + kDepth);
      }
  } else {
#pragma unroll
    for (int s = 0; s < kDepth; ++s)
      if (s < count) fetch(d[s], s);
#pragma unroll 1
    for (int i = 0; i < count; i += kDepth)
#pragma unroll
      for (int s = 0; s < kDepth; ++s)
        if (i + s < count) {
          multiply(d[s]);
          __builtin_amdgcn_sched_barrier(0);
          if (i + s + kDepth < count) fetch(d[s], i + s + kDepth);
        }
  }

  if (!kRoom) fetch_ends();
  // lane (g, m) holds row 16 r + m, columns 16 c + 4 g .. + 3
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int r = 0; r < RT; ++r) *reinterpret_cast<i32x4*>(&part[wave][16 * r + m][16 * c + 4 * g]) = acc[c][r];
  __syncthreads();
  auto sums = [&](int row, int quad) __attribute__((always_inline)) {
    i32x4 v = {};
#pragma unroll
    for (int x = 0; x < kWaves; ++x) v += *reinterpret_cast<const i32x4*>(&part[x][row][4 * quad]);
    return v;
  };
  bool mine = row < it.rows && col < p.n;
  int32_t* units = p.partial + (int64_t)unit * splits * kUnitInts;
  if constexpr (Split) {
    if (tid < it.rows * kQuads) {
      const i32x4 v = sums(tid / kQuads, tid % kQuads);
#pragma unroll
      for (int t = 0; t < 4; ++t) put(units + (int64_t)split * kUnitInts + 4 * tid + t, v[t]);
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // this wave's sums are out
    __syncthreads();
    if (tid == 0) {
      uint32_t* c = p.counters + 16 * unit;
      shared.arrived = __hip_atomic_fetch_add(c, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      if (shared.arrived == (uint32_t)splits - 1)
        __hip_atomic_store(c, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    mine = mine && shared.arrived == (uint32_t)splits - 1;
  }
  if (mine) {
    const int64_t r = it.row + row;
    if constexpr (Fused) {
      uint32_t a = 0;
#pragma unroll
      for (int x = 0; x < kWaves; ++x) a = max(a, shared.most[x][row]);
      step = Quantiser(magnitude<T>(a)).s;
    }
    float residual[4] = {};
    if (!Gated && p.residual != nullptr)
      load_values<T, 4>(static_cast<const uint16_t*>(p.residual) + r * p.ldr + col, residual, p.n - col);
    i32x4 v = {}, u = {};
    if constexpr (Split) {
      const int32_t* from = units + 4 * (row * kQuads + quad);
      for (int s = 0; s < splits; ++s)
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          v[t] += get(from + (int64_t)s * kUnitInts + t);
          if constexpr (Gated) u[t] += get(from + (int64_t)s * kUnitInts + 16 + t);
        }
    } else {
      v = sums(row, quad);
      if constexpr (Gated) u = sums(row, quad + 4);
    }
    float sum[4], up[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      sum[t] = (float)v[t];
      up[t] = (float)u[t];
    }
    with_ending<Gated>(p, [&](auto act) __attribute__((always_inline)) {
      finish<T, Gated, decltype(act)::value, 4>(p, k, (int)r, col, step, sum, up, residual);
    });
  }
  __syncthreads();  // before the next item's sums
}

template <typename T, bool Gated, int C, int RT>
__device__ __forceinline__ void stream_item(const ProductArgs& p, const Item& it, int tile0, int unit, int split,
                                            int splits, Shared& shared) {
  if (splits > 1)
    stream_part<T, Gated, C, RT, false, true>(p, it, tile0, unit, split, splits, shared);
  else
    stream_part<T, Gated, C, RT, false, false>(p, it, tile0, unit, 0, 1, shared);
}

// How many blocks share a unit of work: parts of at least four steps of a wave,
// since a join costs 2 to 3 us, and a step some 0.4 (30 x 16384 x 256: 14 us, not
// split 28; 8 x 8192 x 256: 12.5 and 14.7). What is not split is code of its own
// (30 x 2048 x 7168: 9.2 us, else 9.8).
__device__ __forceinline__ int splits_of(int units, int blocks) {
  return units == 0 || units >= kSplitUnits / 2 ? 1 : max(1, min(kSplitUnits / units, blocks / (4 * kWaves)));
}

template <typename T, bool Gated, int C>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(4, 4)))
void stream_kernel(ProductArgs p) {
  __shared__ __attribute__((aligned(16))) Shared shared;
  const int groups = (packed_tiles<Gated>(p) + C - 1) / C;
  const bool listed = p.lists.counts != nullptr;
  // (at most 2^12 experts by 2^13 groups)
  const int total = (listed ? p.lists.counts[0] : 1) * groups, splits = splits_of(total, p.blocks);
  for (int at = blockIdx.x; at < total * splits; at += gridDim.x) {
    const int u = at / splits, split = at - u * splits;  // (more than one: u < kSplitUnits / 2)
    const int i = u / groups, tile0 = (u - i * groups) * C;
    const Item it = listed ? p.lists.brief[i] : Item{0, 0, p.rows, 0};
    if (it.rows <= 16)
      stream_item<T, Gated, C, 1>(p, it, tile0, u, split, splits, shared);
    else
      stream_item<T, Gated, C, 2>(p, it, tile0, u, split, splits, shared);
  }
}

// The same from the rows as they are, in items of up to kFusedItem of them.
template <typename T, bool Gated, int C>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(4, 4)))
void fused_kernel(ProductArgs p) {
  __shared__ __attribute__((aligned(16))) Shared shared;
  __shared__ Item list[kFusedRows];
  __shared__ int part[kWaves];
  const int t = threadIdx.x;
  int items = 1;
  if (p.offsets != nullptr) {
    items = 0;
    const int end = end_of_rows(p.offsets, p.experts, p.rows);
    for (int e0 = 0; e0 < p.experts; e0 += kThreads) {
      const int e = e0 + t;
      const auto [first, n] = e < p.experts ? range_of(p.offsets, e, end) : Range{0, 0};
      const int m = (n + kFusedItem - 1) / kFusedItem;
      int run = m;
      for (int d = 1; d < kWave; d *= 2) {
        const int v = __shfl_up(run, d);
        run += (t & (kWave - 1)) >= d ? v : 0;
      }
      if ((t & (kWave - 1)) == kWave - 1) part[t / kWave] = run;
      __syncthreads();
      int at = items + run - m;
      for (int w = 0; w < kWaves; ++w) {
        at += w < t / kWave ? part[w] : 0;
        items += part[w];
      }
      for (int i = 0; i < m && at + i < kFusedRows; ++i)
        list[at + i] = Item{e, first + i * kFusedItem, min(n - i * kFusedItem, kFusedItem), 0};
      __syncthreads();
    }
    items = min(items, kFusedRows);
  }
  const int groups = (packed_tiles<Gated>(p) + C - 1) / C, total = items * groups;
  for (int u = blockIdx.x; u < total; u += gridDim.x) {
    const int i = u / groups, tile0 = (u - i * groups) * C;
    Item it{0, 0, p.rows, 0};
    if (p.offsets != nullptr)
      it = Item{__builtin_amdgcn_readfirstlane(list[i].expert), __builtin_amdgcn_readfirstlane(list[i].row),
                __builtin_amdgcn_readfirstlane(list[i].rows), 0};
    stream_part<T, Gated, C, 1, true, false>(p, it, tile0, u, 0, 1, shared);
  }
}

// Two blocks to a CU; four column tiles to each unless that leaves CUs idle (8 x
// 2048 x 7168, 448 column tiles: 7.4 us, by four 8.0; x 10240, 640 of them: 9.7 and
// 8.4).
template <typename T, bool Gated>
static hipError_t launch_typed(const ProductArgs& p, bool fused, hipStream_t stream) {
  const int64_t tiles = (Gated ? 2 : 1) * column_tiles(p.n);
  const int64_t items = p.offsets != nullptr ? most_live(p.rows, p.experts) : 1;
  const dim3 grid(512), block(kThreads);
  const bool narrow = items * tiles <= 512;
  if (fused)
    return launch_kernel(narrow ? fused_kernel<T, Gated, 2> : fused_kernel<T, Gated, 4>, grid, block, stream, p);
  return launch_kernel(narrow ? stream_kernel<T, Gated, 2> : stream_kernel<T, Gated, 4>, grid, block, stream, p);
}

hipError_t launch_stream(int dtype, const ProductArgs& p, bool fused, hipStream_t stream) {
  if (dtype == BLOCK_BF16)
    return p.gated ? launch_typed<BF16, true>(p, fused, stream)
                   : launch_typed<BF16, false>(p, fused, stream);
  return p.gated ? launch_typed<F16, true>(p, fused, stream)
                 : launch_typed<F16, false>(p, fused, stream);
}

}  // namespace experts
