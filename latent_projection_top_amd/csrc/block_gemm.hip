// Matrix products of the layer's operators on the matrix cores.
#include "block_device.h"

#include <algorithm>

namespace block {

// Forward products and dx whose weights the tile kernel's 16-byte loads do not
// fit: rows a multiple of 8 long, for which no copy is kept, at an address
// that is no multiple of 16. (Every other operand is aligned or copied, so dw
// never comes here.) 64 x 64 output tiles, four waves of 32 x 32 each,
// reduction steps of 32 staged element by element through LDS with r
// contiguous: a fifth of the tile kernel's rate (1024 rows of 3584 -> 4096: 176
// us against 36), a ninth at 33 rows (116 against 13.4), whose K it does not
// split.
constexpr int kTile = 64;
constexpr int kStep = 32;
constexpr int kPitch = kStep + 8;  // 16-byte aligned, spreads rows over banks

// Eight consecutive elements of a staged tile: element i at p[i], `count` of
// them inside the matrix, the rest zero.
__device__ __forceinline__ u32x4 load8(const uint16_t* p, int count) {
  if (count >= 8) return reinterpret_cast<const Any16*>(p)->v;
  u32x4 v = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < count) v[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
  return v;
}

// Stage rows i0 .. i0 + 63 (or columns) by r0 .. r0 + 31 of an operand.
template <bool RContig>
__device__ __forceinline__ void stage(uint16_t* lds, const uint16_t* src, int64_t ld, int64_t i0, int64_t ni,
                                      int64_t r0, int64_t nr) {
  const int t = threadIdx.x;
  if constexpr (RContig) {
    const int i = t >> 2, r = 8 * (t & 3);
    const int64_t left = i0 + i < ni ? nr - (r0 + r) : 0;
    const int count = (int)min((int64_t)8, max((int64_t)0, left));
    *reinterpret_cast<u32x4*>(lds + i * kPitch + r) = load8(src + (i0 + i) * ld + r0 + r, count);
  } else {
    const int r = t >> 3, i = 8 * (t & 7);
    const int64_t left = r0 + r < nr ? ni - (i0 + i) : 0;
    const int count = (int)min((int64_t)8, max((int64_t)0, left));
    const u32x4 v = load8(src + (r0 + r) * ld + i0 + i, count);
#pragma unroll
    for (int j = 0; j < 8; ++j) lds[(i + j) * kPitch + r] = (uint16_t)(v[j >> 1] >> (16 * (j & 1)));
  }
}

template <typename T, int Mode>
__global__ __launch_bounds__(256) void gemm_narrow_kernel(GemmArgs p) {
  constexpr bool kBContig = Mode == kDx;
  constexpr int kB = Mode == kGated ? 2 : 1;
  __shared__ __attribute__((aligned(16))) uint16_t sa[kTile * kPitch];
  __shared__ __attribute__((aligned(16))) uint16_t sb[kB][kTile * kPitch];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, g = lane >> 4, m = lane & 15;
  const int64_t row0 = (int64_t)blockIdx.y * kTile;
  const int col0 = blockIdx.x * kTile;
  const int wr = 32 * (wave >> 1), wc = 32 * (wave & 1);
  f32x4 acc[kB][2][2] = {};
  for (int s = 0; s < p.segments; ++s) {
    const uint16_t* a = static_cast<const uint16_t*>(p.a[s]);
    for (int64_t r0 = 0; r0 < p.red; r0 += kStep) {
      stage<true>(sa, a, p.lda, row0, p.m, r0, p.red);
#pragma unroll
      for (int b = 0; b < kB; ++b)
        stage<kBContig>(sb[b], static_cast<const uint16_t*>(p.b[Mode == kGated ? b : s]), p.ldb, col0, p.n, r0,
                        p.red);
      __syncthreads();
      u32x4 av[2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
        av[i] = *reinterpret_cast<const u32x4*>(sa + (wr + 16 * i + m) * kPitch + 8 * g);
#pragma unroll
      for (int b = 0; b < kB; ++b)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const u32x4 bv = *reinterpret_cast<const u32x4*>(sb[b] + (wc + 16 * j + m) * kPitch + 8 * g);
#pragma unroll
          for (int i = 0; i < 2; ++i) acc[b][i][j] = T::mfma(bv, av[i], acc[b][i][j]);
        }
      __syncthreads();
    }
  }
  // columns on the matrix instruction's row side: a lane holds four
  // consecutive columns of one row
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float v[4], u[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        v[t] = acc[0][i][j][t];
        u[t] = acc[kB - 1][i][j][t];
      }
      epilogue<T, Mode, 4>(p, 0, row0 + wr + 16 * i + m, col0 + wc + 16 * j + 4 * g, v, u);
    }
}

template <typename T>
static hipError_t launch_narrow(Mode mode, const GemmArgs& p, hipStream_t stream) {
  const dim3 grid((p.n + kTile - 1) / kTile, (unsigned)((p.m + kTile - 1) / kTile));
  switch (mode) {
    case kLinear: return launch_kernel(gemm_narrow_kernel<T, kLinear>, grid, dim3(256), stream, p);
    case kGated: return launch_kernel(gemm_narrow_kernel<T, kGated>, grid, dim3(256), stream, p);
    default: return launch_kernel(gemm_narrow_kernel<T, kDx>, grid, dim3(256), stream, p);
  }
}

// Joins the splits' FP32 sums in split order and ends the product.
template <typename T, int Mode>
__global__ __launch_bounds__(256) void gemm_join_kernel(GemmArgs p, int splits, const float* partial) {
  const int64_t pn = (p.n + 3) & ~3, quads = pn / 4;
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int planes = Mode == kGated ? 2 : p.outputs;
  const int64_t plane = p.m * pn;
  if (id >= quads * p.m * (Mode == kGated ? 1 : planes)) return;
  const int which = (int)(id / (quads * p.m));
  const int64_t q = id - which * quads * p.m;
  const int64_t row = q / quads;
  const int col = (int)(q - row * quads) * 4;
  const float* d = partial + which * plane + row * pn + col;
  f32x4 vs = {0.f, 0.f, 0.f, 0.f}, us = vs;
  #pragma unroll 4
  for (int s = 0; s < splits; ++s) {
    vs += *reinterpret_cast<const f32x4*>(d);
    if (Mode == kGated) us += *reinterpret_cast<const f32x4*>(d + plane);
    d += planes * plane;
  }
  float v[4], u[4];
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    v[t] = vs[t];
    u[t] = us[t];
  }
  epilogue<T, Mode, 4>(p, which, row, col, v, u);
}

template <typename T>
static hipError_t join_typed(Mode mode, const GemmArgs& p, int splits, const float* partial, hipStream_t stream) {
  const int64_t items = (int64_t)((p.n + 3) / 4) * p.m * (mode == kGated ? 1 : p.outputs);
  const dim3 grid((unsigned)((items + 255) / 256));
  switch (mode) {
    case kLinear: return launch_kernel(gemm_join_kernel<T, kLinear>, grid, dim3(256), stream, p, splits, partial);
    case kGated: return launch_kernel(gemm_join_kernel<T, kGated>, grid, dim3(256), stream, p, splits, partial);
    case kDx: return launch_kernel(gemm_join_kernel<T, kDx>, grid, dim3(256), stream, p, splits, partial);
    default: return launch_kernel(gemm_join_kernel<T, kDw>, grid, dim3(256), stream, p, splits, partial);
  }
}

hipError_t launch_gemm_join(int dtype, Mode mode, const GemmArgs& p, int splits, const float* partial,
                            hipStream_t stream) {
  return dtype == BLOCK_BF16 ? join_typed<BF16>(mode, p, splits, partial, stream)
                             : join_typed<F16>(mode, p, splits, partial, stream);
}

// Whether the tile kernel can read every operand (contiguous lengths that are
// no multiple of 8 come as padded copies).
static bool tileable(const GemmArgs& p) {
  uintptr_t bits = 0;
  for (int i = 0; i < 2; ++i)
    bits |= reinterpret_cast<uintptr_t>(p.a[i]) | reinterpret_cast<uintptr_t>(p.b[i]);
  return (bits & 15) == 0 && ((p.lda | p.ldb) & 7) == 0;
}

bool gemm_streams(Mode mode, int64_t m, int64_t n, int64_t red) {
  return mode != kDw && m <= kStreamRows && red >= 8 && n >= 8;
}

// 64 MB at most: sums that large cost more on their way out and back than a
// split gains.
size_t gemm_partial_bytes(Mode mode, int64_t m, int n, int64_t red, int segments, int outputs) {
  const size_t row = (size_t)((n + 3) & ~3) * 4 * (mode == kGated ? 2 : outputs), most = (size_t)64 << 20;
  size_t bytes = 0;
  if (gemm_streams(mode, 1, n, red)) {
    const size_t splits = most_stream_splits(mode, n, red, segments);
    if (splits > 1) bytes = splits * (size_t)std::min<int64_t>(m, kStreamRows) * row;
  }
  if (!gemm_streams(mode, m, n, red)) {  // the tile kernel too
    const size_t splits = most_tile_splits(red, segments), plane = (size_t)m * row;
    // dw is of this size in every call; the others may be of any up to it
    const size_t tile = mode == kDw ? std::min(splits, most / plane) * plane : std::min(splits * plane, most);
    if (splits > 1 && (mode != kDw || tile > plane)) bytes = std::max(bytes, tile);
  }
  return bytes;
}

hipError_t launch_gemm(int dtype, Mode mode, const GemmArgs& p, const Workspace& ws, hipStream_t stream) {
  if (gemm_streams(mode, p.m, p.n, p.red))
    return launch_gemm_stream(dtype, mode, p, ws, stream);
  if (tileable(p))
    return launch_gemm_tile(dtype, mode, p, plan_tiles(mode, p, ws.partial_bytes), ws.partial, stream);
  return dtype == BLOCK_BF16 ? launch_narrow<BF16>(mode, p, stream) : launch_narrow<F16>(mode, p, stream);
}

// ------------------------------------------------------------- elementwise --

struct Copies {
  Copy c[3];
  int64_t end[3];  // pieces of 8 values, counted through
};

__global__ __launch_bounds__(256) void copy_kernel(Copies p) {
  for (int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x; at < p.end[2]; at += (int64_t)gridDim.x * 256) {
    const int k = at < p.end[0] ? 0 : at < p.end[1] ? 1 : 2;
    const Copy& c = p.c[k];
    const int64_t id = k > 0 ? at - p.end[k - 1] : at;
    const int64_t per_row = (c.len + 7) >> 3;
    const int64_t row = id / per_row;
    const int col = (int)(id - row * per_row) * 8;
    const u32x4 v = load8(static_cast<const uint16_t*>(c.src) + row * c.ld + col, c.len - col);
    *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(c.dst) + id * 8) = v;
  }
}

hipError_t launch_copies(const Copy* copies, int count, hipStream_t stream) {
  Copies p{};
  int64_t end = 0;
  for (int k = 0; k < 3; ++k) {
    if (k < count) {
      p.c[k] = copies[k];
      end += copies[k].rows * ((copies[k].len + 7) >> 3);
    }
    p.end[k] = end;
  }
  if (end == 0) return hipSuccess;
  // A launch has fewer than 2^32 threads, and 2^20 rows of 131072 values are
  // 2^34 pieces: beyond 2^28 threads each takes several.
  const int64_t blocks = std::min<int64_t>((end + 255) / 256, 1 << 20);
  return launch_kernel(copy_kernel, dim3((unsigned)blocks), dim3(256), stream, p);
}

// The first half of a backward pass: out[k] = dy * s[k], rounded to the
// products' type, and where dbias is wanted the column sums of the unrounded
// out[0] (of dy itself where there is no s). One pass over its inputs, bound
// by HBM: a thread owns eight columns and walks down every gridDim.y-th row.
struct ScaleArgs {
  const void* dy;
  const void* s[2];
  void* out[2];
  float* partial;  // [gridDim.y][n rounded up to 8], or NULL
  int64_t dy_stride, ld, rows;
  int n;
};

template <typename T, int Count, bool Sum>
__global__ __launch_bounds__(256) void scale_kernel(ScaleArgs p) {
  const int col = 8 * (blockIdx.x * 256 + threadIdx.x);
  if (col >= p.n) return;
  const int count = min(8, p.n - col);
  float sum[8] = {};
#pragma unroll 2
  for (int64_t row = blockIdx.y; row < p.rows; row += gridDim.y) {
    const u32x4 dy = load8(static_cast<const uint16_t*>(p.dy) + row * p.dy_stride + col, count);
    float d[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) d[i] = T::load((uint16_t)(dy[i >> 1] >> (16 * (i & 1))));
#pragma unroll
    for (int k = 0; k < Count; ++k) {
      const u32x4 s = load8(static_cast<const uint16_t*>(p.s[k]) + row * p.n + col, count);
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = d[i] * T::load((uint16_t)(s[i >> 1] >> (16 * (i & 1))));
        if (Sum) sum[i] += v[i];
      }
      u32x4 o;
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = T::store2(v[2 * i], v[2 * i + 1]);
      // the row stride is a multiple of 8: the last piece pads with zeros
      if (p.out[k] != nullptr)
        *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p.out[k]) + row * p.ld + col) = o;
    }
    if (Sum && Count == 0)
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] += d[i];
  }
  if (Sum) {
    float* d = p.partial + (int64_t)blockIdx.y * ((p.n + 7) & ~7) + col;
    *reinterpret_cast<f32x4*>(d) = f32x4{sum[0], sum[1], sum[2], sum[3]};
    *reinterpret_cast<f32x4*>(d + 4) = f32x4{sum[4], sum[5], sum[6], sum[7]};
  }
}

// Adds the blocks' column sums: 32 columns per block, 32 slices of the
// blocks, each slice and then the slices in order.
template <typename T>
__global__ __launch_bounds__(256) void column_join_kernel(const float* partial, int blocks, int n, uint16_t* dst) {
  __shared__ f32x4 part[32][8];
  const int64_t ld = (n + 7) & ~7;
  const int q = threadIdx.x & 7, slice = threadIdx.x >> 3;
  const int c = (blockIdx.x * 8 + q) * 4;
  f32x4 s = {0.f, 0.f, 0.f, 0.f};
  if (c < n)
#pragma unroll 8
    for (int b = slice; b < blocks; b += 32) s += *reinterpret_cast<const f32x4*>(partial + (int64_t)b * ld + c);
  part[slice][q] = s;
  __syncthreads();
  const int t = threadIdx.x, col = blockIdx.x * 32 + t;
  if (t >= 32 || col >= n) return;
  float v = 0.f;
#pragma unroll
  for (int i = 0; i < 32; ++i) v += part[i][t >> 2][t & 3];
  dst[col] = T::store(v);
}

// Blocks of rows: enough to fill the CUs, and for sums no more (each writes a
// row of partial sums).
static int scale_blocks(int64_t rows, int n, bool sum) {
  const int64_t across = ((int64_t)n + 2047) / 2048;
  int64_t most = (sum ? 1024 : 2048) / across;
  if (most < 1) most = 1;
  return (int)(rows < most ? (rows > 0 ? rows : 1) : most);
}

template <typename T>
static hipError_t scale_typed(const ScaleArgs& p, int count, void* dbias, hipStream_t stream) {
  const int blocks = scale_blocks(p.rows, p.n, dbias != nullptr);
  const dim3 grid((p.n + 2047) / 2048, blocks);
  hipError_t e;
  if (dbias == nullptr)
    e = launch_kernel(count == 2 ? scale_kernel<T, 2, false> : scale_kernel<T, 1, false>, grid, dim3(256), stream, p);
  else
    e = launch_kernel(count == 1 ? scale_kernel<T, 1, true> : scale_kernel<T, 0, true>, grid, dim3(256), stream, p);
  if (e != hipSuccess || dbias == nullptr) return e;
  return launch_kernel(column_join_kernel<T>, dim3((p.n + 31) / 32), dim3(256), stream,
                       static_cast<const float*>(p.partial), blocks, p.n, static_cast<uint16_t*>(dbias));
}

hipError_t launch_scale(int dtype, const void* dy, int64_t dy_stride, const void* const* s, int count,
                        void* const* out, int64_t ld, int64_t rows, int n, void* dbias, float* partial,
                        hipStream_t stream) {
  ScaleArgs p{};
  p.dy = dy;
  for (int k = 0; k < count; ++k) {
    p.s[k] = s[k];
    p.out[k] = out[k];
  }
  p.partial = partial;
  p.dy_stride = dy_stride;
  p.ld = ld;
  p.rows = rows;
  p.n = n;
  return dtype == BLOCK_BF16 ? scale_typed<BF16>(p, count, dbias, stream)
                             : scale_typed<F16>(p, count, dbias, stream);
}

size_t column_sum_bytes(int64_t rows, int n) {
  return (size_t)scale_blocks(rows, n, true) * ((n + 7) & ~7) * 4;
}

}  // namespace block
