// Matrix products of few rows (up to 32): every weight is used for a handful
// of rows, so the time is the weights' way from HBM, and the kernel is built
// around keeping many of their bytes in flight.
//
// A wave takes 128 columns by 32 of the reduction at a time, straight into
// registers (8 loads of 16 bytes per lane, the next step's under way while
// this one is multiplied), and multiplies on the matrix cores with the rows
// padded to 16. The eight waves of a block take its steps in turn and their
// sums meet in LDS; with few column tiles the reduction is also split over
// blocks and joined by a second kernel.
//
// Weights with contiguous columns ([K][N], forward): lane (g, m) loads rows
// 8 g .. 8 g + 7 of columns 8 m .. 8 m + 7 (256-byte segments) and transposes
// the 8 x 8 block with v_perm_b32: fragment c holds columns 8 m + c.
// Weights with a contiguous reduction (backward, W^T): lane (g, m) loads
// 8 values of columns 8 m + c, c = 0..7, which are the fragments as they are.
#include "block_device.h"

namespace block {

constexpr int kCols = 128;   // columns of a tile
constexpr int kRed = 32;     // reduction of a step
constexpr int kWaves = 8;
constexpr int kPart = kCols + 4;  // floats of a row of partial sums in LDS

// `v` moved down by d elements of 16 bits, zeros from above (d >= 8: all).
__device__ __forceinline__ u32x4 drop_low(u32x4 v, int d) {
  if (d & 4) v = u32x4{v[2], v[3], 0, 0};
  if (d & 2) v = u32x4{v[1], v[2], v[3], 0};
  if (d & 1)
    v = u32x4{v[0] >> 16 | v[1] << 16, v[1] >> 16 | v[2] << 16, v[2] >> 16 | v[3] << 16, v[3] >> 16};
  return d >= 8 ? u32x4{0, 0, 0, 0} : v;
}

__device__ __forceinline__ u32x4 load16(const uint16_t* p) { return reinterpret_cast<const Any16*>(p)->v; }

template <typename T, int Mode, int RT>
__global__ __launch_bounds__(64 * kWaves) void gemm_stream_kernel(GemmArgs p, int splits, float* partial) {
  constexpr bool kTurn = Mode != kDx;                  // weights need the transpose
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
    u32x4 x[RT];
  };
  // Everything a lane loads is inside the matrices: columns past the end
  // repeat the last eight (or the last one), the reduction past the end is
  // clamped here and taken out in `trim`.
  auto fetch = [&](Step& d, int i) {
    const int s = s0 + i * kTeam;
    const int seg = s >= per_seg ? 1 : 0;
    const int k0 = (s - seg * per_seg) * kRed;
    const int k = k0 + 8 * g;
    const uint16_t* w = static_cast<const uint16_t*>(p.b[Mode == kGated ? wave / kTeam : seg]);
    if constexpr (kTurn) {
      const int col = min(col0 + 8 * m, p.n - 8);
#pragma unroll
      for (int r = 0; r < 8; ++r) d.w[r] = load16(w + (int64_t)min(k + r, red - 1) * p.ldb + col);
    } else {
#pragma unroll
      for (int c = 0; c < 8; ++c)
        d.w[c] = load16(w + (int64_t)min(col0 + 8 * m + c, p.n - 1) * p.ldb + min(k, red - 8));
    }
    const uint16_t* x = static_cast<const uint16_t*>(p.a[seg]) + min(k, red - 8);
#pragma unroll
    for (int r = 0; r < RT; ++r) d.x[r] = load16(x + min((int64_t)(16 * r + m), p.m - 1) * p.lda);
  };

  f32x4 acc[8][RT] = {};
  auto multiply = [&](Step& d, int i) {
    const int s = s0 + i * kTeam;
    const int ks = s >= per_seg ? s - per_seg : s;
    if (ks == per_seg - 1) {  // the reduction may end inside: zeros from there
      const int k = ks * kRed + 8 * g;
      const int over = min(max(k - (red - 8), 0), 8);
#pragma unroll
      for (int r = 0; r < RT; ++r) d.x[r] = drop_low(d.x[r], over);
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        if constexpr (kTurn)
          d.w[r] = k + r < red ? d.w[r] : u32x4{0, 0, 0, 0};
        else
          d.w[r] = drop_low(d.w[r], over);
      }
    }
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      u32x4 f;
      if constexpr (kTurn) {
        constexpr uint32_t kLow = 0x05040100, kHigh = 0x07060302;
#pragma unroll
        for (int q = 0; q < 4; ++q)
          f[q] = __builtin_amdgcn_perm(d.w[2 * q + 1][c >> 1], d.w[2 * q][c >> 1], (c & 1) ? kHigh : kLow);
      } else {
        f = d.w[c];
      }
#pragma unroll
      for (int r = 0; r < RT; ++r) acc[c][r] = T::mfma(f, d.x[r], acc[c][r]);
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

  // lane (g, m) holds row 16 r + m; acc[c][r][t] is column 8 (4 g + t) + c
  const int64_t pn = (p.n + 3) & ~3;
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    float* d = &part[wave][16 * r + m][32 * g];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      *reinterpret_cast<f32x4*>(d + 8 * t) = f32x4{acc[0][r][t], acc[1][r][t], acc[2][r][t], acc[3][r][t]};
      *reinterpret_cast<f32x4*>(d + 8 * t + 4) = f32x4{acc[4][r][t], acc[5][r][t], acc[6][r][t], acc[7][r][t]};
    }
  }
  __syncthreads();
  for (int id = threadIdx.x; id < (int)p.m * 16; id += 64 * kWaves) {
    const int row = id >> 4, run = id & 15;
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
        *reinterpret_cast<f32x4*>(d + 4 * q) = f32x4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
        if (Mode == kGated)
          *reinterpret_cast<f32x4*>(d + p.m * pn + 4 * q) =
              f32x4{u[4 * q], u[4 * q + 1], u[4 * q + 2], u[4 * q + 3]};
      }
    } else {
      epilogue<T, Mode, 8>(p, 0, row, col, v, u);
    }
  }
}

template <typename T, int Mode>
static hipError_t launch_rows(const GemmArgs& p, int splits, float* partial, hipStream_t stream) {
  const dim3 grid((p.n + kCols - 1) / kCols, splits), block(64 * kWaves);
  if (p.m <= 16) return launch_kernel(gemm_stream_kernel<T, Mode, 1>, grid, block, stream, p, splits, partial);
  return launch_kernel(gemm_stream_kernel<T, Mode, 2>, grid, block, stream, p, splits, partial);
}

template <typename T>
static hipError_t launch_typed(Mode mode, const GemmArgs& p, int splits, float* partial, hipStream_t stream) {
  switch (mode) {
    case kLinear: return launch_rows<T, kLinear>(p, splits, partial, stream);
    case kGated: return launch_rows<T, kGated>(p, splits, partial, stream);
    default: return launch_rows<T, kDx>(p, splits, partial, stream);
  }
}

hipError_t launch_gemm_stream(int dtype, Mode mode, const GemmArgs& p, float* partial, size_t partial_bytes,
                              hipStream_t stream) {
  const int64_t tiles = (p.n + kCols - 1) / kCols;
  const int64_t steps = (p.red + kRed - 1) / kRed * p.segments;
  const int team = mode == kGated ? kWaves / 2 : kWaves;
  const int64_t plane = (int64_t)p.m * ((p.n + 3) & ~3) * 4 * (mode == kGated ? 2 : 1);
  // a block per CU, but a step at least for every wave
  int64_t splits = tiles >= 256 ? 1 : (p.m <= 16 ? (256 + tiles - 1) / tiles : 256 / tiles);
  splits = splits < steps / team ? splits : steps / team;
  splits = splits < (int64_t)partial_bytes / plane ? splits : (int64_t)partial_bytes / plane;
  splits = splits < 1 ? 1 : (splits > 64 ? 64 : splits);
  const hipError_t e = dtype == BLOCK_BF16 ? launch_typed<BF16>(mode, p, (int)splits, partial, stream)
                                           : launch_typed<F16>(mode, p, (int)splits, partial, stream);
  if (e != hipSuccess || splits == 1) return e;
  return launch_gemm_join(dtype, mode, p, (int)splits, partial, stream);
}

}  // namespace block
