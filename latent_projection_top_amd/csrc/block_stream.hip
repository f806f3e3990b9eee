// Matrix products of few rows (up to 32): every weight is used for a handful
// of rows, so the time is the weights' way from HBM, and the kernel is built
// around keeping many of their bytes in flight.
//
// A wave takes 8 KB of weights at a time, straight into registers (8 loads of
// 16 bytes per lane, the next step's under way while this one is multiplied),
// and multiplies on the matrix cores with the rows padded to 16. The eight
// waves of a block take its steps in turn and their sums meet in LDS. With
// few column tiles the reduction is also split over blocks: their FP32 sums
// go through the workspace and are added in split order, by the last block of
// a tile to arrive where they are few (Join), by a second kernel where they
// are many.
//
// Weights with contiguous columns ([K][N], forward): a step is 128 columns by
// 32 of the reduction. Lane (g, m) loads rows 8 g .. 8 g + 7 of columns 8 m ..
// 8 m + 7 (256-byte segments) and transposes the 8 x 8 block with v_perm_b32:
// fragment c holds columns 8 m + c.
// Weights with a contiguous reduction (backward, W^T): a step is 64 columns by
// 64 of the reduction. Lane (g, m) loads values 16 g .. 16 g + 15 of columns
// 4 m + c, c = 0..3 (whole 128-byte lines; with half the reduction and twice
// the columns, 64-byte segments, one row of 7168 -> 7168 took 25.1 us instead of
// 23.3), which are two fragments as they are: the order of a reduction is
// free as long as both operands have it.
//
//   1 row of gated 7168 x 7168: 41 us (5.0 TB/s); 20 rows of gated 7168 x 2048:
//   14 us and 4 for the join; 8 rows of 2048 x 7168: 8.4-10 us. Around the
//   stream, a start of about 3 us and a join of 2 to 5.
#include "block_device.h"

#include <algorithm>

namespace block {

constexpr int kWaves = 8;
constexpr int stream_cols(int mode) { return mode == kDx ? 64 : 128; }  // of a step and tile
constexpr int stream_red(int mode) { return mode == kDx ? 64 : 32; }    // of a step

// `v` moved down by d elements of 16 bits, zeros from above (d >= 8: all).
__device__ __forceinline__ u32x4 drop_low(u32x4 v, int d) {
  if (d & 4) v = u32x4{v[2], v[3], 0, 0};
  if (d & 2) v = u32x4{v[1], v[2], v[3], 0};
  if (d & 1)
    v = u32x4{v[0] >> 16 | v[1] << 16, v[1] >> 16 | v[2] << 16, v[2] >> 16 | v[3] << 16, v[3] >> 16};
  return d >= 8 ? u32x4{0, 0, 0, 0} : v;
}

__device__ __forceinline__ u32x4 load16(const uint16_t* p) { return reinterpret_cast<const Any16*>(p)->v; }

// Partial sums between blocks of one launch: relaxed device-scope atomics,
// which go past the XCDs' L2s both ways, so that no fence has to write a
// whole L2 back. A block waits for its stores before it counts itself in.
__device__ __forceinline__ void put4(float* p, float a, float b, float c, float d) {
  auto pair = [](float lo, float hi) { return (uint64_t)__float_as_uint(hi) << 32 | __float_as_uint(lo); };
  uint64_t* q = reinterpret_cast<uint64_t*>(p);
  __hip_atomic_store(q, pair(a, b), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __hip_atomic_store(q + 1, pair(c, d), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void get2(const float* p, float& a, float& b) {
  const uint64_t v = __hip_atomic_load(reinterpret_cast<uint64_t*>(const_cast<float*>(p)), __ATOMIC_RELAXED,
                                       __HIP_MEMORY_SCOPE_AGENT);
  a = __uint_as_float((uint32_t)v);
  b = __uint_as_float((uint32_t)(v >> 32));
}

template <typename T, int Mode, int RT, bool Join>
__global__ __launch_bounds__(64 * kWaves) void gemm_stream_kernel(GemmArgs p, int splits, float* partial,
                                                                  uint32_t* counters) {
  constexpr bool kTurn = Mode != kDx;  // weights need the transpose
  constexpr int kCols = stream_cols(Mode), kRed = stream_red(Mode);
  constexpr int kMine = kCols / 16;        // columns of a lane, kMine m + c
  constexpr int kHalves = kRed / 32;       // MFMAs deep
  constexpr int kPart = kCols + 4;         // floats of a row of partial sums
  constexpr int kTeam = Mode == kGated ? kWaves / 2 : kWaves;  // waves of one matrix
  __shared__ __attribute__((aligned(16))) float part[kWaves][16 * RT][kPart];

  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, g = lane >> 4, m = lane & 15;
  const int tile = blockIdx.x, split = blockIdx.y;
  const int col0 = tile * kCols;
  const int per_seg = (int)((p.red + kRed - 1) / kRed);
  const int all = per_seg * p.segments;
  const int s0 = (int)((int64_t)all * split / splits) + wave % kTeam;
  const int s1 = (int)((int64_t)all * (split + 1) / splits);
  const int count = s1 > s0 ? (s1 - s0 + kTeam - 1) / kTeam : 0;
  const int red = (int)p.red;

  struct Step {
    u32x4 w[8];
    u32x4 x[RT][kHalves];
  };
  // Everything a lane loads is inside the matrices: columns past the end
  // repeat the last eight (or the last one), the reduction past the end is
  // clamped here and taken out in `trim`.
  auto fetch = [&](Step& d, int i) {
    const int s = s0 + i * kTeam;
    const int seg = s >= per_seg ? 1 : 0;
    const int k0 = (s - seg * per_seg) * kRed;
    const int k = k0 + 8 * kHalves * g;
    const uint16_t* w = static_cast<const uint16_t*>(p.b[Mode == kGated ? wave / kTeam : seg]);
    if constexpr (kTurn) {
      const int col = min(col0 + 8 * m, p.n - 8);
#pragma unroll
      for (int r = 0; r < 8; ++r) d.w[r] = load16(w + (int64_t)min(k + r, red - 1) * p.ldb + col);
    } else {
#pragma unroll
      for (int c = 0; c < kMine; ++c)
#pragma unroll
        for (int h = 0; h < kHalves; ++h)
          d.w[c * kHalves + h] =
              load16(w + (int64_t)min(col0 + kMine * m + c, p.n - 1) * p.ldb + min(k + 8 * h, red - 8));
    }
    const uint16_t* x = static_cast<const uint16_t*>(p.a[seg]);
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int h = 0; h < kHalves; ++h)
        d.x[r][h] = load16(x + min((int64_t)(16 * r + m), p.m - 1) * p.lda + min(k + 8 * h, red - 8));
  };

  f32x4 acc[kMine][RT] = {};
  auto multiply = [&](Step& d, int i) {
    const int s = s0 + i * kTeam;
    const int ks = s >= per_seg ? s - per_seg : s;
    if (ks == per_seg - 1) {  // the reduction may end inside: zeros from there
      const int k = ks * kRed + 8 * kHalves * g;
#pragma unroll
      for (int h = 0; h < kHalves; ++h) {
        const int over = min(max(k + 8 * h - (red - 8), 0), 8);
#pragma unroll
        for (int r = 0; r < RT; ++r) d.x[r][h] = drop_low(d.x[r][h], over);
        if constexpr (!kTurn)
#pragma unroll
          for (int c = 0; c < kMine; ++c) d.w[c * kHalves + h] = drop_low(d.w[c * kHalves + h], over);
      }
      if constexpr (kTurn)
#pragma unroll
        for (int r = 0; r < 8; ++r) d.w[r] = k + r < red ? d.w[r] : u32x4{0, 0, 0, 0};
    }
#pragma unroll
    for (int c = 0; c < kMine; ++c)
#pragma unroll
      for (int h = 0; h < kHalves; ++h) {
        u32x4 f;
        if constexpr (kTurn) {
          constexpr uint32_t kLow = 0x05040100, kHigh = 0x07060302;
#pragma unroll
          for (int q = 0; q < 4; ++q)
            f[q] = __builtin_amdgcn_perm(d.w[2 * q + 1][c >> 1], d.w[2 * q][c >> 1], (c & 1) ? kHigh : kLow);
        } else {
          f = d.w[c * kHalves + h];
        }
#pragma unroll
        for (int r = 0; r < RT; ++r) acc[c][r] = T::mfma(f, d.x[r][h], acc[c][r]);
      }
  };

  if (count > 0) {
    Step d0, d1;
    fetch(d0, 0);
    int i = 0;
#pragma unroll 1
    for (; i + 2 < count; i += 2) {
      fetch(d1, i + 1);
      __builtin_amdgcn_sched_barrier(0);
      multiply(d0, i);
      fetch(d0, i + 2);
      __builtin_amdgcn_sched_barrier(0);
      multiply(d1, i + 1);
    }
    if (i + 1 < count) {
      fetch(d1, i + 1);
      __builtin_amdgcn_sched_barrier(0);
      multiply(d0, i);
      multiply(d1, i + 1);
    } else {
      multiply(d0, i);
    }
  }

  // lane (g, m) holds row 16 r + m; acc[c][r][t] is column kMine (4 g + t) + c
  const int64_t pn = (p.n + 3) & ~3;
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    float* d = &part[wave][16 * r + m][4 * kMine * g];
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int c = 0; c < kMine; c += 4)
        *reinterpret_cast<f32x4*>(d + kMine * t + c) =
            f32x4{acc[c][r][t], acc[c + 1][r][t], acc[c + 2][r][t], acc[c + 3][r][t]};
  }
  __syncthreads();
  for (int id = threadIdx.x; id < (int)p.m * (kCols / 8); id += 64 * kWaves) {
    const int row = id / (kCols / 8), run = id % (kCols / 8);
    const int col = col0 + 8 * run;
    if (col >= p.n) continue;
    float v[8] = {}, u[8] = {};
#pragma unroll
    for (int w = 0; w < kTeam; ++w)
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        v[c] += part[w][row][8 * run + c];
        if (Mode == kGated) u[c] += part[kTeam + w][row][8 * run + c];
      }
    if (kTurn && col + 8 > p.n) {
      // this run's lane loaded the last eight columns, n - 8 + c: bring
      // column col + c to place c
      const int d = col - (p.n - 8);
#pragma unroll
      for (int c = 0; c < 8; ++c)
#pragma unroll
        for (int e = c + 1; e < 8; ++e)
          if (e == c + d) {
            v[c] = v[e];
            u[c] = u[e];
          }
    }
    if (splits > 1) {
      constexpr int kPlanes = Mode == kGated ? 2 : 1;
      float* d = partial + ((int64_t)split * kPlanes * p.m + row) * pn + col;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        if (col + 4 * q >= p.n) break;
        if constexpr (Join) {
          put4(d + 4 * q, v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
          if (Mode == kGated) put4(d + p.m * pn + 4 * q, u[4 * q], u[4 * q + 1], u[4 * q + 2], u[4 * q + 3]);
        } else {
          *reinterpret_cast<f32x4*>(d + 4 * q) = f32x4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
          if (Mode == kGated)
            *reinterpret_cast<f32x4*>(d + p.m * pn + 4 * q) =
                f32x4{u[4 * q], u[4 * q + 1], u[4 * q + 2], u[4 * q + 3]};
        }
      }
    } else {
      epilogue<T, Mode, 8>(p, 0, row, col, v, u);
    }
  }
  if constexpr (Join) {
    // The tile's last block adds the splits' sums. Its counter goes back to
    // zero for the next call.
    __shared__ uint32_t arrived;
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // this wave's sums are out
    __syncthreads();
    if (threadIdx.x == 0) {
      uint32_t* c = counters + 16 * tile;
      arrived = __hip_atomic_fetch_add(c, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      if (arrived == (uint32_t)splits - 1) __hip_atomic_store(c, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    if (arrived != (uint32_t)splits - 1) return;
    constexpr int kPlanes = Mode == kGated ? 2 : 1;
    for (int id = threadIdx.x; id < (int)p.m * (kCols / 4); id += 64 * kWaves) {
      const int row = id / (kCols / 4), col = col0 + 4 * (id % (kCols / 4));
      if (col >= p.n) continue;
      const float* d = partial + (int64_t)row * pn + col;
      float v[4] = {}, u[4] = {};
      // eight splits' loads in flight at a time
#pragma unroll 1
      for (int s = 0; s < splits; s += 8) {
        float x[8][4], y[8][4];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float* e = d + (int64_t)min(s + q, splits - 1) * kPlanes * p.m * pn;
          get2(e, x[q][0], x[q][1]);
          get2(e + 2, x[q][2], x[q][3]);
          if (Mode == kGated) {
            get2(e + p.m * pn, y[q][0], y[q][1]);
            get2(e + p.m * pn + 2, y[q][2], y[q][3]);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (s + q < splits)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              v[c] += x[q][c];
              if (Mode == kGated) u[c] += y[q][c];
            }
      }
      epilogue<T, Mode, 4>(p, 0, row, col, v, u);
    }
  }
}

template <typename T, int Mode>
static hipError_t launch_rows(const GemmArgs& p, int splits, bool join, float* partial, uint32_t* counters,
                              hipStream_t stream) {
  constexpr int kCols = stream_cols(Mode);
  const dim3 grid((p.n + kCols - 1) / kCols, splits), block(64 * kWaves);
  const bool one = p.m <= 16;
  if (join)
    return launch_kernel(one ? gemm_stream_kernel<T, Mode, 1, true> : gemm_stream_kernel<T, Mode, 2, true>, grid,
                         block, stream, p, splits, partial, counters);
  return launch_kernel(one ? gemm_stream_kernel<T, Mode, 1, false> : gemm_stream_kernel<T, Mode, 2, false>, grid,
                       block, stream, p, splits, partial, counters);
}

template <typename T>
static hipError_t launch_typed(Mode mode, const GemmArgs& p, int splits, bool join, float* partial,
                               uint32_t* counters, hipStream_t stream) {
  switch (mode) {
    case kLinear: return launch_rows<T, kLinear>(p, splits, join, partial, counters, stream);
    case kGated: return launch_rows<T, kGated>(p, splits, join, partial, counters, stream);
    default: return launch_rows<T, kDx>(p, splits, join, partial, counters, stream);
  }
}

struct StreamPlan {
  int splits;
  bool join;  // by the last block of each tile
};

constexpr int kMaxSplits = 64;

int most_stream_splits(Mode mode, int n, int64_t red, int segments) {
  const int64_t tiles = (n + stream_cols(mode) - 1) / stream_cols(mode);
  const int64_t steps = (red + stream_red(mode) - 1) / stream_red(mode) * segments;
  return (int)std::max<int64_t>(1, std::min({(int64_t)kMaxSplits, steps, 256 / tiles}));
}

// At most a block per CU: a second round costs another start and end (16 rows
// of 3584 x 7168: 4 splits, 224 blocks, 15.3 us; 5 splits, 280 blocks, 20.4;
// 9 splits, 504 blocks, 17.2). Within that, the split whose modelled time is
// least: the weights at 5.2 TB/s, or 0.12 us (backward 0.2) for each step of a
// block if that is more; 0.6 us (1.0) for each of a wave's steps in turn; 3.0
// us and 0.07 a split for a join by the last block, or 5.3 for one by a second
// kernel and the sums twice at 4 TB/s (1000 x 776, 1 row: 6.6 us unsplit, 5.6
// with 8 splits; 512 x 512: 4.0 unsplit, 4.8 with 8).
// The last block joins up to 8 rows of sums (8 rows of 2048 x 7168, 4 splits:
// 10.7 us against 11.4; 1 row of gated 3584 x 2048, 16 splits: 10.4 against
// 12.3); beyond, its one CU takes longer than a second kernel on all of them
// (16 rows of 3584 x 7168, 4 splits: 16.3 against 15.3).
static StreamPlan plan_stream(Mode mode, const GemmArgs& p, size_t partial_bytes) {
  const int cols = stream_cols(mode), red = stream_red(mode);
  const int64_t tiles = (p.n + cols - 1) / cols;
  const int most = most_stream_splits(mode, p.n, p.red, p.segments);
  const int64_t steps = (p.red + red - 1) / red * p.segments;
  const int planes = mode == kGated ? 2 : 1, team = kWaves / planes;
  const double plane = (double)p.m * ((p.n + 3) & ~3) * 4 * planes;
  const double bytes = (double)tiles * steps * planes * (cols * red * 2);
  const bool join = p.m * planes <= 8;
  const double per_step = mode == kDx ? 0.2 : 0.12, per_turn = mode == kDx ? 1.0 : 0.6;
  StreamPlan best{1, false};
  double best_t = 0;
  for (int s = 1; s <= most; ++s) {
    if (s > 1 && plane * s > (double)partial_bytes) break;
    const int64_t block_steps = (steps + s - 1) / s;
    const double t = std::max(bytes / 5.2e6, per_step * (double)(block_steps * planes)) +
                     per_turn * (double)((block_steps + team - 1) / team) + (s == 1 ? 0.0 : join ? 3.0 + 0.07 * s : 5.3 + 2.0 * s * plane / 4e6);
    if (s == 1 || t <= best_t) {
      best = StreamPlan{s, join && s > 1};
      best_t = t;
    }
  }
  return best;
}

hipError_t launch_gemm_stream(int dtype, Mode mode, const GemmArgs& p, const Workspace& ws, hipStream_t stream) {
  const StreamPlan t = plan_stream(mode, p, ws.partial_bytes);
  const hipError_t e = dtype == BLOCK_BF16
                           ? launch_typed<BF16>(mode, p, t.splits, t.join, ws.partial, ws.counters, stream)
                           : launch_typed<F16>(mode, p, t.splits, t.join, ws.partial, ws.counters, stream);
  if (e != hipSuccess || t.splits == 1 || t.join) return e;
  return launch_gemm_join(dtype, mode, p, t.splits, ws.partial, stream);
}

}  // namespace block
