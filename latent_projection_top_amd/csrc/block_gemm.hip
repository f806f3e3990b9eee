// Matrix products of the layer's operators on the matrix cores.
#include "block_device.h"

namespace block {

// Products that the tile kernel's 16-byte loads do not fit: weights whose
// rows are multiples of 8 long, for which no copy is kept, at an address that
// is no multiple of 16. 64 x 64 output tiles, four waves of
// 32 x 32 each, reduction steps of 32 staged element by element through LDS
// with r contiguous; right for everything, at about a fifth of the tile
// kernel's rate.
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
  constexpr bool kAContig = Mode != kDw, kBContig = Mode == kDx;
  constexpr int kB = Mode == kGated ? 2 : 1;
  __shared__ __attribute__((aligned(16))) uint16_t sa[kTile * kPitch];
  __shared__ __attribute__((aligned(16))) uint16_t sb[kB][kTile * kPitch];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, g = lane >> 4, m = lane & 15;
  const int64_t row0 = (int64_t)blockIdx.y * kTile;
  const int col0 = blockIdx.x * kTile;
  const int which = blockIdx.z;
  const int wr = 32 * (wave >> 1), wc = 32 * (wave & 1);
  f32x4 acc[kB][2][2] = {};
  for (int s = 0; s < p.segments; ++s) {
    const uint16_t* a = static_cast<const uint16_t*>(p.a[s]);
    for (int64_t r0 = 0; r0 < p.red; r0 += kStep) {
      stage<kAContig>(sa, a, p.lda, row0, p.m, r0, p.red);
#pragma unroll
      for (int b = 0; b < kB; ++b)
        stage<kBContig>(sb[b], static_cast<const uint16_t*>(p.b[Mode == kGated ? b : s + which]), p.ldb, col0,
                        p.n, r0, p.red);
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
      epilogue<T, Mode, 4>(p, which, row0 + wr + 16 * i + m, col0 + wc + 16 * j + 4 * g, v, u);
    }
}

template <typename T>
static hipError_t launch_narrow(Mode mode, const GemmArgs& p, hipStream_t stream) {
  const dim3 grid((p.n + kTile - 1) / kTile, (unsigned)((p.m + kTile - 1) / kTile), mode == kDw ? p.outputs : 1);
  switch (mode) {
    case kLinear: return launch_kernel(gemm_narrow_kernel<T, kLinear>, grid, dim3(256), stream, p);
    case kGated: return launch_kernel(gemm_narrow_kernel<T, kGated>, grid, dim3(256), stream, p);
    case kDx: return launch_kernel(gemm_narrow_kernel<T, kDx>, grid, dim3(256), stream, p);
    default: return launch_kernel(gemm_narrow_kernel<T, kDw>, grid, dim3(256), stream, p);
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

// Whether the tile kernel can read every operand.
static int64_t lengths(Mode mode, const GemmArgs& p) {
  return (mode == kDw ? p.m : p.red) | (mode == kDx ? p.red : p.n);
}

static bool tileable(Mode mode, const GemmArgs& p) {
  uintptr_t bits = 0;
  for (int i = 0; i < 2; ++i)
    bits |= reinterpret_cast<uintptr_t>(p.a[i]) | reinterpret_cast<uintptr_t>(p.b[i]);
  return (bits & 15) == 0 && ((p.lda | p.ldb) & 7) == 0 && (p.padded || (lengths(mode, p) & 7) == 0);
}

bool gemm_streams(Mode mode, int64_t m, int64_t n, int64_t red) {
  return mode != kDw && m <= kStreamRows && red >= 8 && n >= 8;
}

size_t gemm_partial_bytes(Mode mode, int64_t m, int n, int outputs) {
  const size_t plane = (size_t)m * ((n + 3) & ~3) * 4 * (mode == kGated ? 2 : outputs);
  // only products of few tiles are split
  const size_t most = (size_t)64 << 20;
  return plane * kMaxSplits < most ? plane * kMaxSplits : most;
}

hipError_t launch_gemm(int dtype, Mode mode, const GemmArgs& p, const Workspace& ws, hipStream_t stream) {
  if (gemm_streams(mode, p.m, p.n, p.red))
    return launch_gemm_stream(dtype, mode, p, ws, stream);
  if (tileable(mode, p))
    return launch_gemm_tile(dtype, mode, p, plan_tiles(mode, p, ws.partial_bytes), ws.partial, stream);
  return dtype == BLOCK_BF16 ? launch_narrow<BF16>(mode, p, stream) : launch_narrow<F16>(mode, p, stream);
}

// ------------------------------------------------------------- elementwise --

struct Copies {
  Copy c[3];
  int64_t end[3];  // pieces of 8 values, counted through
};

__global__ __launch_bounds__(256) void copy_kernel(Copies p) {
  int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (id >= p.end[2]) return;
  const int k = id < p.end[0] ? 0 : id < p.end[1] ? 1 : 2;
  const Copy& c = p.c[k];
  if (k > 0) id -= p.end[k - 1];
  const int64_t per_row = (c.len + 7) >> 3;
  const int64_t row = id / per_row;
  const int col = (int)(id - row * per_row) * 8;
  const u32x4 v = load8(static_cast<const uint16_t*>(c.src) + row * c.ld + col, c.len - col);
  *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(c.dst) + id * 8) = v;
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
  return launch_kernel(copy_kernel, dim3((unsigned)((end + 255) / 256)), dim3(256), stream, p);
}

struct ScaleArgs {
  const void* dy;
  const void* s[2];
  void* out[2];
  int64_t dy_stride, ld;
  int n;
};

template <typename T, int Count>
__global__ __launch_bounds__(256) void scale_kernel(ScaleArgs p) {
  const int64_t row = blockIdx.y;
  const int col = 8 * (blockIdx.x * 256 + threadIdx.x);
  if (col >= p.n) return;
  const int count = min(8, p.n - col);
  const u32x4 dy = load8(static_cast<const uint16_t*>(p.dy) + row * p.dy_stride + col, count);
#pragma unroll
  for (int k = 0; k < Count; ++k) {
    const u32x4 s = load8(static_cast<const uint16_t*>(p.s[k]) + row * p.n + col, count);
    u32x4 o = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float v = T::load((uint16_t)(dy[i >> 1] >> (16 * (i & 1)))) *
                      T::load((uint16_t)(s[i >> 1] >> (16 * (i & 1))));
      o[i >> 1] |= (uint32_t)T::store(v) << (16 * (i & 1));
    }
    // the row stride is a multiple of 8, so the last piece may run past n
    *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p.out[k]) + row * p.ld + col) = o;
  }
}

template <typename T>
static hipError_t scale_typed(const ScaleArgs& p, int count, int64_t rows, hipStream_t stream) {
  // rows in launches of at most 65535 (the grid's y limit)
  for (int64_t r = 0; r < rows; r += 65535) {
    ScaleArgs q = p;
    q.dy = static_cast<const uint16_t*>(p.dy) + r * p.dy_stride;
    for (int k = 0; k < count; ++k) {
      q.s[k] = static_cast<const uint16_t*>(p.s[k]) + r * p.n;
      q.out[k] = static_cast<uint16_t*>(p.out[k]) + r * p.ld;
    }
    const dim3 grid((p.n + 2047) / 2048, (unsigned)(rows - r < 65535 ? rows - r : 65535));
    const hipError_t e = count == 2 ? launch_kernel(scale_kernel<T, 2>, grid, dim3(256), stream, q)
                                    : launch_kernel(scale_kernel<T, 1>, grid, dim3(256), stream, q);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_scale(int dtype, const void* dy, int64_t dy_stride, const void* const* s, int count,
                        void* const* out, int64_t ld, int64_t rows, int n, hipStream_t stream) {
  ScaleArgs p{dy, {s[0], count > 1 ? s[1] : nullptr}, {out[0], count > 1 ? out[1] : nullptr}, dy_stride, ld, n};
  return dtype == BLOCK_BF16 ? scale_typed<BF16>(p, count, rows, stream)
                             : scale_typed<F16>(p, count, rows, stream);
}

// Column sums: blocks of 64 columns, four row lanes each, the four joined in
// a fixed order.
template <typename T>
__global__ __launch_bounds__(256) void column_sum_kernel(const uint16_t* src, int64_t ld, int64_t rows, int n,
                                                         uint16_t* dst) {
  __shared__ float red[256];
  const int col = blockIdx.x * 64 + (threadIdx.x & 63);
  float s = 0.f;
  if (col < n)
    for (int64_t r = threadIdx.x >> 6; r < rows; r += 4) s += T::load(src[r * ld + col]);
  red[threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.x < 64 && col < n)
    dst[col] = T::store((red[threadIdx.x] + red[threadIdx.x + 64]) +
                        (red[threadIdx.x + 128] + red[threadIdx.x + 192]));
}

hipError_t launch_column_sum(int dtype, const void* src, int64_t ld, int64_t rows, int n, void* dst,
                             float* partial, hipStream_t stream) {
  (void)partial;
  const dim3 grid((n + 63) / 64);
  const uint16_t* s = static_cast<const uint16_t*>(src);
  uint16_t* d = static_cast<uint16_t*>(dst);
  return dtype == BLOCK_BF16 ? launch_kernel(column_sum_kernel<BF16>, grid, dim3(256), stream, s, ld, rows, n, d)
                             : launch_kernel(column_sum_kernel<F16>, grid, dim3(256), stream, s, ld, rows, n, d);
}

size_t column_sum_bytes(int64_t, int) { return 0; }

}  // namespace block
