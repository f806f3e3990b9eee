// Layer norm, forward and backward: bound by HBM (large) or by the latency of
// one load, one or two reductions and one store (few rows).
//
// A row lives in the registers of `Lanes` threads from its one load to its
// store, in 16-byte pieces: thread l holds pieces l and l + Lanes. The mean is
// summed first and the variance from the centred values, so nothing cancels
// for rows far from zero. Blocks stay and walk over rows, which keeps weight
// and bias in registers (re-read per row they would be four times the row's
// own bytes from L2) and lets the next row's loads fly during the reductions.
// Backward, each thread also keeps the FP32 sums of its columns' dweight and
// dbias over the block's rows; a second kernel adds the blocks' sums in block
// order.
//   16384 x 7168 BF16: forward 82-97 us (4.8-5.7 TB/s), backward 140-153
//   (4.6-5.0; a copy reaches 5.06-5.14); 1 x 7168: 2.7 us forward, 4.0 backward.
#include "block_device.h"

#include <cmath>

namespace block {

// ------------------------------------------------------------------ pieces --

// One 16-byte piece of a row (`E` elements), or a single element where the
// row is narrower than a piece.
template <typename T, int E>
struct Piece {
  u32x4 v;
  __device__ __forceinline__ void load(const typename T::raw* p) {
    if constexpr (E == 1) {
      if constexpr (sizeof(typename T::raw) == 4)
        v[0] = __float_as_uint(*p);
      else
        v[0] = *p;
    } else {
      v = reinterpret_cast<const Any16*>(p)->v;
    }
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (sizeof(typename T::raw) == 4) return __uint_as_float(v[i]);
    else return T::load((uint16_t)(v[i >> 1] >> (16 * (i & 1))));
  }
  static __device__ __forceinline__ void store(typename T::raw* p, const float (&f)[E]) {
    if constexpr (E == 1) {
      *p = T::store(f[0]);
    } else if constexpr (sizeof(typename T::raw) == 4) {
      reinterpret_cast<Any16*>(p)->v = u32x4{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                                             __float_as_uint(f[3])};
    } else {
      u32x4 w;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = T::store2(f[2 * i], f[2 * i + 1]);
      reinterpret_cast<Any16*>(p)->v = w;
    }
  }
};

// E parameters of runtime type from element i on; `def` without any.
template <int E>
__device__ __forceinline__ void load_params(const void* p, int i, int dtype, float def, float (&f)[E]) {
#pragma unroll
  for (int e = 0; e < E; ++e) f[e] = def;
  if (p == nullptr) return;
  if (dtype == BLOCK_F32) {
#pragma unroll
    for (int e = 0; e < E; ++e) f[e] = static_cast<const float*>(p)[i + e];
  } else if (dtype == BLOCK_BF16) {
#pragma unroll
    for (int e = 0; e < E; ++e) f[e] = BF16::load(static_cast<const uint16_t*>(p)[i + e]);
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) f[e] = F16::load(static_cast<const uint16_t*>(p)[i + e]);
  }
}

struct __attribute__((packed, aligned(4))) AnyF4 { f32x4 v; };

// ----------------------------------------------------------------- reduction --

template <int Ctrl>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), Ctrl, 0xF, 0xF, true));
}

// Sum over a row of 16 lanes, in every lane (rotations within the row).
__device__ __forceinline__ float sum16(float v) {
  v = dpp_add<0x128>(v);
  v = dpp_add<0x124>(v);
  v = dpp_add<0x122>(v);
  return dpp_add<0x121>(v);
}

__device__ __forceinline__ float sum64(float v) {
  v = sum16(v);
  auto lane = [&](int l) { return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), l)); };
  return (lane(0) + lane(16)) + (lane(32) + lane(48));
}

// Sum of N values over the Lanes threads of a row, in a fixed order, returned
// to all of them. slot: LDS for Lanes / 64 x N floats; a slot may be written
// again only after a later reduction's barrier.
template <int Lanes, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float* slot) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = Lanes == 16 ? sum16(v[i]) : sum64(v[i]);
  if constexpr (Lanes > 64) {
    constexpr int kW = Lanes / 64;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) slot[i * kW + (threadIdx.x >> 6)] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < kW; ++w) s += slot[i * kW + w];
      v[i] = s;
    }
  }
}

// ------------------------------------------------------------------- forward --

// A thread's pieces of a row. The last piece of a row whose width is no
// multiple of E starts early, to end with the row; its first `skip` elements
// belong to the piece before and count for nothing here.
template <int Lanes, int P, int E>
struct Columns {
  int start[P];
  int skip[P];  // E: no piece
  __device__ __forceinline__ Columns(int lane, int width) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int c = (lane + Lanes * i) * E;
      start[i] = min(c, width - E);
      skip[i] = min(c - start[i], E);
    }
  }
};

template <typename T, int Lanes, int P, int E>
__global__ __launch_bounds__(Lanes < 256 ? 256 : Lanes) void norm_kernel(NormArgs p) {
  typedef typename T::raw raw;
  constexpr int kThreads = Lanes < 256 ? 256 : Lanes;
  constexpr int kRows = kThreads / Lanes;  // rows of a block at a time
  constexpr bool kKeep = P <= 2;           // parameters stay in registers
  __shared__ float red[2][Lanes > 64 ? Lanes / 64 : 1];
  const Columns<Lanes, P, E> col(threadIdx.x % Lanes, p.width);
  const int64_t step = (int64_t)gridDim.x * kRows;
  const float n = (float)p.width;
  float w[P][E], b[P][E];
  if (kKeep) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      load_params(p.weight, col.start[i], p.param_dtype, 1.f, w[i]);
      load_params(p.bias, col.start[i], p.param_dtype, 0.f, b[i]);
    }
  }
  Piece<T, E> x[P], next[P];
  auto fetch = [&](Piece<T, E>(&d)[P], int64_t row) {
    // rows past the end repeat the last one: no branch around the loads
    const raw* src = static_cast<const raw*>(p.x) + min(row, p.rows - 1) * p.ldx;
#pragma unroll
    for (int i = 0; i < P; ++i) d[i].load(src + col.start[i]);
  };
  const int64_t first = (int64_t)blockIdx.x * kRows + threadIdx.x / Lanes;
  fetch(x, first);
  // every thread of a block makes the same number of turns
  for (int64_t r0 = (int64_t)blockIdx.x * kRows; r0 < p.rows; r0 += step) {
    const int64_t row = r0 + threadIdx.x / Lanes;
    if (kKeep) fetch(next, row + step);
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
      for (int e = 0; e < E; ++e) s[0] += e >= col.skip[i] ? x[i].get(e) : 0.f;
    row_sum<Lanes>(s, red[0]);
    const float mean = s[0] / n;  // (times 1 / n would leave a constant row off its mean)
    float v[1] = {0.f};
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float d = e >= col.skip[i] ? x[i].get(e) - mean : 0.f;
        v[0] += d * d;
      }
    row_sum<Lanes>(v, red[1]);
    const float rstd = 1.f / sqrtf(v[0] / n + p.eps);
    if (row < p.rows) {
      raw* y = static_cast<raw*>(p.y) + row * p.ldy;
#pragma unroll
      for (int i = 0; i < P; ++i) {
        if (col.skip[i] >= E) continue;
        if (!kKeep) {
          load_params(p.weight, col.start[i], p.param_dtype, 1.f, w[i]);
          load_params(p.bias, col.start[i], p.param_dtype, 0.f, b[i]);
        }
        float o[E];
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = (x[i].get(e) - mean) * rstd * w[i][e] + b[i][e];
        // (an early piece stores the elements it shares with the one before
        // it a second time, with the same value)
        Piece<T, E>::store(y + col.start[i], o);
      }
      if (p.mean != nullptr && threadIdx.x % Lanes == 0) {
        p.mean[row] = mean;
        p.rstd[row] = rstd;
      }
    }
    if (kKeep) {
#pragma unroll
      for (int i = 0; i < P; ++i) x[i] = next[i];
    } else {
      fetch(x, row + step);
    }
  }
}

// ------------------------------------------------------------------ backward --

template <typename T, int Lanes, int P, int E>
__global__ __launch_bounds__(Lanes < 256 ? 256 : Lanes) void norm_backward_kernel(NormArgs p) {
  typedef typename T::raw raw;
  constexpr int kThreads = Lanes < 256 ? 256 : Lanes;
  constexpr int kRows = kThreads / Lanes;
  // next row and weights in registers, if 128 (of 1024 threads) hold them
  constexpr bool kKeep = Lanes * P * E <= 8192;
  __shared__ float red[2][Lanes > 64 ? 2 * (Lanes / 64) : 2];
  const int lane = threadIdx.x % Lanes, group = threadIdx.x / Lanes;
  const Columns<Lanes, P, E> col(lane, p.width);
  const int64_t step = (int64_t)gridDim.x * kRows;
  const float n = (float)p.width;
  float w[P][E], dw[P][E] = {}, db[P][E] = {};
  if (kKeep)
#pragma unroll
    for (int i = 0; i < P; ++i) load_params(p.weight, col.start[i], p.param_dtype, 1.f, w[i]);
  Piece<T, E> x[P], dy[P], nx[P], ndy[P];
  float mean, rstd, nmean, nrstd;
  auto fetch = [&](Piece<T, E>(&dx_)[P], Piece<T, E>(&dd)[P], float& m, float& r, int64_t row) {
    row = min(row, p.rows - 1);
    const raw* sx = static_cast<const raw*>(p.x) + row * p.ldx;
    const raw* sd = static_cast<const raw*>(p.dy) + row * p.lddy;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      dx_[i].load(sx + col.start[i]);
      dd[i].load(sd + col.start[i]);
    }
    m = p.mean[row];
    r = p.rstd[row];
  };
  int turn = 0;
  if (p.rows > 0) fetch(x, dy, mean, rstd, (int64_t)blockIdx.x * kRows + group);
  for (int64_t r0 = (int64_t)blockIdx.x * kRows; r0 < p.rows; r0 += step) {
    const int64_t row = r0 + group;
    if (kKeep) fetch(nx, ndy, nmean, nrstd, row + step);
    const bool live = row < p.rows;
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < P; ++i) {
      if (!kKeep) load_params(p.weight, col.start[i], p.param_dtype, 1.f, w[i]);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const bool in = live && e >= col.skip[i];
        const float d = dy[i].get(e), xh = (x[i].get(e) - mean) * rstd;
        db[i][e] += in ? d : 0.f;
        dw[i][e] += in ? d * xh : 0.f;
        const float g = in ? w[i][e] * d : 0.f;
        s[0] += g;
        s[1] += in ? g * xh : 0.f;
      }
    }
    if (p.dx != nullptr) {
      row_sum<Lanes>(s, red[turn & 1]);
      ++turn;
      const float c1 = s[0] / n, c2 = s[1] / n;
      if (live) {
        raw* dx = static_cast<raw*>(p.dx) + row * p.lddx;
#pragma unroll
        for (int i = 0; i < P; ++i) {
          if (col.skip[i] >= E) continue;
          if (!kKeep) load_params(p.weight, col.start[i], p.param_dtype, 1.f, w[i]);
          float o[E];
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const float xh = (x[i].get(e) - mean) * rstd;
            o[e] = rstd * (w[i][e] * dy[i].get(e) - c1 - xh * c2);
          }
          Piece<T, E>::store(dx + col.start[i], o);
        }
      }
    }
    if (kKeep) {
#pragma unroll
      for (int i = 0; i < P; ++i) {
        x[i] = nx[i];
        dy[i] = ndy[i];
      }
      mean = nmean;
      rstd = nrstd;
    } else {
      fetch(x, dy, mean, rstd, row + step);
    }
  }
  if (p.dweight == nullptr && p.dbias == nullptr) return;
  // the block's sums: groups joined in LDS in group order, then out; those of
  // a block alone are the result
  const bool alone = gridDim.x == 1;
  auto result = [&](int k, int c, float v) {
    void* dst = k == 0 ? p.dweight : p.dbias;
    if (dst != nullptr) store_param(dst, c, p.param_dtype, v);
  };
  const int64_t wp = (p.width + 3) & ~3;
  float* out = p.partial + (int64_t)blockIdx.x * 2 * wp;
  if constexpr (kRows == 1) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      float* o = out + col.start[i];
      if (alone && E >= 4 && col.skip[i] == 0 && p.param_dtype == BLOCK_F32) {
#pragma unroll
        for (int e = 0; e + 4 <= E; e += 4) {
          const int c = col.start[i] + e;
          if (p.dweight)
            reinterpret_cast<AnyF4*>(static_cast<float*>(p.dweight) + c)->v =
                f32x4{dw[i][e], dw[i][e + 1], dw[i][e + 2], dw[i][e + 3]};
          if (p.dbias)
            reinterpret_cast<AnyF4*>(static_cast<float*>(p.dbias) + c)->v =
                f32x4{db[i][e], db[i][e + 1], db[i][e + 2], db[i][e + 3]};
        }
        continue;
      }
      if (alone) {
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (e >= col.skip[i]) {
            result(0, col.start[i] + e, dw[i][e]);
            result(1, col.start[i] + e, db[i][e]);
          }
        continue;
      }
      if (E >= 4 && col.skip[i] == 0) {
#pragma unroll
        for (int e = 0; e + 4 <= E; e += 4) {
          *reinterpret_cast<f32x4*>(o + e) = f32x4{dw[i][e], dw[i][e + 1], dw[i][e + 2], dw[i][e + 3]};
          *reinterpret_cast<f32x4*>(o + wp + e) = f32x4{db[i][e], db[i][e + 1], db[i][e + 2], db[i][e + 3]};
        }
        continue;
      }
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (e >= col.skip[i]) {
          o[e] = dw[i][e];
          o[wp + e] = db[i][e];
        }
    }
  } else {
    __shared__ float join[kRows][Lanes * P * E];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < P; ++i)
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (e >= col.skip[i]) join[group][col.start[i] + e] = k == 0 ? dw[i][e] : db[i][e];
      __syncthreads();
      for (int c = threadIdx.x; c < p.width; c += kThreads) {
        float s = 0.f;
#pragma unroll
        for (int r = 0; r < kRows; ++r) s += join[r][c];
        if (alone)
          result(k, c, s);
        else
          out[k * wp + c] = s;
      }
    }
  }
}

// dweight and dbias from the blocks' sums: 32 columns per block, 32 slices of
// the blocks, each slice in order and then the slices pairwise, which rounds a
// sum five times on its way where adding them in order would 31 times (RMS of
// dbias over 517 rows of FP32: 0.9e-7 against 1.25e-7).
__global__ __launch_bounds__(256) void norm_join_kernel(NormArgs p, int blocks) {
  __shared__ f32x4 part[32][8];
  const int64_t wp = (p.width + 3) & ~3;
  const int q = threadIdx.x & 7, slice = threadIdx.x >> 3;
  const int c = (blockIdx.x * 8 + q) * 4;
  const int k = blockIdx.y;
  f32x4 s = {0.f, 0.f, 0.f, 0.f};
  if (c < wp) {
    const float* src = p.partial + k * wp + c;
#pragma unroll 8
    for (int b = slice; b < blocks; b += 32) s += *reinterpret_cast<const f32x4*>(src + (int64_t)b * 2 * wp);
  }
  part[slice][q] = s;
  __syncthreads();
  const int t = threadIdx.x;
  void* dst = k == 0 ? p.dweight : p.dbias;
  if (t >= 32 || dst == nullptr) return;
  const int cc = blockIdx.x * 32 + t;
  if (cc >= p.width) return;
  float v[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = part[i][t >> 2][t & 3];
#pragma unroll
  for (int half = 16; half > 0; half >>= 1)
#pragma unroll
    for (int i = 0; i < half; ++i) v[i] += v[i + half];
  store_param(dst, cc, p.param_dtype, v[0]);
}

// ---------------------------------------------------------------- wide rows --

// Rows that registers do not hold (over 4096 pieces): a block of 1024 threads
// reads the row once per pass.
__device__ __forceinline__ float wide_sum(float v, float* red) {
  v = sum64(v);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < 16; ++w) s += red[w];
  __syncthreads();
  return s;
}

template <typename T>
__global__ __launch_bounds__(1024) void norm_wide_kernel(NormArgs p) {
  __shared__ float red[16];
  const int64_t row = blockIdx.x;
  const typename T::raw* x = static_cast<const typename T::raw*>(p.x) + row * p.ldx;
  typename T::raw* y = static_cast<typename T::raw*>(p.y) + row * p.ldy;
  float s = 0.f;
  for (int i = threadIdx.x; i < p.width; i += 1024) s += T::load(x[i]);
  const float mean = wide_sum(s, red) / (float)p.width;
  float v = 0.f;
  for (int i = threadIdx.x; i < p.width; i += 1024) {
    const float d = T::load(x[i]) - mean;
    v += d * d;
  }
  const float rstd = 1.f / sqrtf(wide_sum(v, red) / (float)p.width + p.eps);
  for (int i = threadIdx.x; i < p.width; i += 1024) {
    const float w = p.weight ? load_param(p.weight, i, p.param_dtype) : 1.f;
    const float b = p.bias ? load_param(p.bias, i, p.param_dtype) : 0.f;
    y[i] = T::store((T::load(x[i]) - mean) * rstd * w + b);
  }
  if (p.mean != nullptr && threadIdx.x == 0) {
    p.mean[row] = mean;
    p.rstd[row] = rstd;
  }
}

template <typename T>
__global__ __launch_bounds__(1024) void norm_wide_dx_kernel(NormArgs p) {
  __shared__ float red[16];
  const int64_t row = blockIdx.x;
  const typename T::raw* x = static_cast<const typename T::raw*>(p.x) + row * p.ldx;
  const typename T::raw* dy = static_cast<const typename T::raw*>(p.dy) + row * p.lddy;
  typename T::raw* dx = static_cast<typename T::raw*>(p.dx) + row * p.lddx;
  const float mean = p.mean[row], rstd = p.rstd[row];
  float s1 = 0.f, s2 = 0.f;
  for (int i = threadIdx.x; i < p.width; i += 1024) {
    const float w = p.weight ? load_param(p.weight, i, p.param_dtype) : 1.f;
    const float g = w * T::load(dy[i]);
    s1 += g;
    s2 += g * ((T::load(x[i]) - mean) * rstd);
  }
  s1 = wide_sum(s1, red) / (float)p.width;
  s2 = wide_sum(s2, red) / (float)p.width;
  for (int i = threadIdx.x; i < p.width; i += 1024) {
    const float w = p.weight ? load_param(p.weight, i, p.param_dtype) : 1.f;
    const float xh = (T::load(x[i]) - mean) * rstd;
    dx[i] = T::store(rstd * (w * T::load(dy[i]) - s1 - xh * s2));
  }
}

// Blocks of 64 columns, sixteen row lanes each, joined in a fixed order.
template <typename T>
__global__ __launch_bounds__(1024) void norm_wide_dparam_kernel(NormArgs p) {
  __shared__ float part[2][16][64];
  const int c = threadIdx.x & 63, lane = threadIdx.x >> 6;
  const int col = blockIdx.x * 64 + c;
  float sw = 0.f, sb = 0.f;
  if (col < p.width) {
#pragma unroll 4
    for (int64_t r = lane; r < p.rows; r += 16) {
      const float dy = T::load(static_cast<const typename T::raw*>(p.dy)[r * p.lddy + col]);
      const float x = T::load(static_cast<const typename T::raw*>(p.x)[r * p.ldx + col]);
      sb += dy;
      sw += dy * ((x - p.mean[r]) * p.rstd[r]);
    }
  }
  part[0][lane][c] = sw;
  part[1][lane][c] = sb;
  __syncthreads();
  if (lane > 1 || col >= p.width) return;
  void* dst = lane == 0 ? p.dweight : p.dbias;
  if (dst == nullptr) return;
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) s += part[lane][i][c];
  store_param(dst, col, p.param_dtype, s);
}

// ------------------------------------------------------------------ launches --

// Calls f(Lanes, P, E) with the fewest threads that hold a row in at most two
// pieces each (four from 2048 pieces on); false: registers do not hold it.
template <int E, typename F>
static bool with_layout(int width, F f) {
  const int pieces = (width + E - 1) / E;
  auto c = [&](auto lanes, auto p) { f(lanes, p, std::integral_constant<int, E>{}); return true; };
  using std::integral_constant;
  if (pieces <= 32) return c(integral_constant<int, 16>{}, integral_constant<int, 2>{});
  if (pieces <= 128) return c(integral_constant<int, 64>{}, integral_constant<int, 2>{});
  if (pieces <= 512) return c(integral_constant<int, 256>{}, integral_constant<int, 2>{});
  if (pieces <= 1024) return c(integral_constant<int, 512>{}, integral_constant<int, 2>{});
  if (pieces <= 2048) return c(integral_constant<int, 1024>{}, integral_constant<int, 2>{});
  if (pieces <= 4096) return c(integral_constant<int, 1024>{}, integral_constant<int, 4>{});
  return false;
}

// (most: no more than that many pieces)
template <typename T, typename F>
static bool with_row_layout(int width, int most, F f) {
  constexpr int kE = 16 / sizeof(typename T::raw);
  if (width < kE) {
    f(std::integral_constant<int, 16>{}, std::integral_constant<int, 1>{}, std::integral_constant<int, 1>{});
    return true;
  }
  return (width + kE - 1) / kE <= most && with_layout<kE>(width, f);
}
// Backward, rows of more than 2048 pieces keep twice as many sums per thread
// as its registers hold (2048 x 20000: 374 us spilling, 120 by the wide
// kernels).
constexpr int kForwardPieces = 4096, kBackwardPieces = 2048;

// Blocks that stay, at most `most` of them, each with whole groups of rows.
static int64_t norm_blocks(int64_t rows, int lanes, int64_t most) {
  const int64_t group = (lanes < 256 ? 256 : lanes) / lanes;
  const int64_t turns = (rows + group - 1) / group;
  return turns < most ? turns : most;
}

// Forward: the threads that two blocks of 512 per CU come to.
static int64_t forward_blocks(int64_t rows, int lanes) {
  return norm_blocks(rows, lanes, 256 * 1024 / (lanes < 256 ? 256 : lanes));
}

// Backward: every block also writes 8 bytes per column, which the join reads
// again. With B blocks a row takes about 1.2 us of its block, and the sums 16
// B width bytes at 5 TB/s, together least at B = sqrt(375000 rows / width);
// 512 threads per CU saturate HBM (16384 x 7168: 142 us for 705 MB). 256 rows
// of 7168: 12.5 + 3 us with 116 blocks, 12 + 4.5 with 256.
static int64_t backward_blocks(int64_t rows, int lanes, int width) {
  const int64_t most = 256 * 512 / (lanes < 256 ? 256 : lanes);
  const int64_t best = (int64_t)std::sqrt(375000.0 * (double)rows / (double)width) + 1;
  const int64_t blocks = norm_blocks(rows, lanes, best < most ? best : most);
  // one block needs no join: for narrow rows up to four turns of it cost less
  // than a launch (80 x 80, both passes: 19.5 us of eager calls against 23.8)
  return lanes < 256 && norm_blocks(rows, lanes, 5) < 5 ? 1 : blocks;
}

template <typename T>
static hipError_t norm_typed(const NormArgs& p, hipStream_t stream) {
  hipError_t e = hipSuccess;
  const bool held = with_row_layout<T>(p.width, kForwardPieces, [&](auto lanes, auto pieces, auto el) {
    constexpr int L = decltype(lanes)::value, P = decltype(pieces)::value, E = decltype(el)::value;
    e = launch_kernel(norm_kernel<T, L, P, E>, dim3((unsigned)forward_blocks(p.rows, L)),
                      dim3(L < 256 ? 256 : L), stream, p);
  });
  return held ? e : launch_kernel(norm_wide_kernel<T>, dim3((unsigned)p.rows), dim3(1024), stream, p);
}

template <typename T>
static hipError_t norm_backward_typed(const NormArgs& p, hipStream_t stream) {
  const bool params = p.dweight != nullptr || p.dbias != nullptr;
  hipError_t e = hipSuccess;
  int64_t blocks = 0;
  const bool held = with_row_layout<T>(p.width, kBackwardPieces, [&](auto lanes, auto pieces, auto el) {
    constexpr int L = decltype(lanes)::value, P = decltype(pieces)::value, E = decltype(el)::value;
    blocks = backward_blocks(p.rows, L, p.width);
    if constexpr (P <= 2)
      if (blocks > 0)
        e = launch_kernel(norm_backward_kernel<T, L, P, E>, dim3((unsigned)blocks), dim3(L < 256 ? 256 : L), stream, p);
  });
  if (e != hipSuccess) return e;
  if (held)
    return params && blocks != 1 ? launch_kernel(norm_join_kernel, dim3((p.width + 31) / 32, 2), dim3(256), stream, p, (int)blocks)
                  : hipSuccess;
  if (p.dx != nullptr && p.rows > 0)
    e = launch_kernel(norm_wide_dx_kernel<T>, dim3((unsigned)p.rows), dim3(1024), stream, p);
  if (e != hipSuccess || !params) return e;
  return launch_kernel(norm_wide_dparam_kernel<T>, dim3((p.width + 63) / 64), dim3(1024), stream, p);
}

hipError_t launch_norm(int dtype, const NormArgs& p, hipStream_t stream) {
  if (dtype == BLOCK_F32) return norm_typed<F32>(p, stream);
  if (dtype == BLOCK_F16) return norm_typed<F16>(p, stream);
  return norm_typed<BF16>(p, stream);
}

hipError_t launch_norm_backward(int dtype, const NormArgs& p, hipStream_t stream) {
  if (dtype == BLOCK_F32) return norm_backward_typed<F32>(p, stream);
  if (dtype == BLOCK_F16) return norm_backward_typed<F16>(p, stream);
  return norm_backward_typed<BF16>(p, stream);
}

template <typename T>
static size_t backward_bytes(int64_t rows, int width) {
  size_t bytes = 0;
  with_row_layout<T>(width, kBackwardPieces, [&](auto lanes, auto, auto) {
    bytes = (size_t)backward_blocks(rows, decltype(lanes)::value, width) * 2 * ((width + 3) & ~3) * 4;
  });
  return bytes;
}

size_t norm_backward_bytes(int dtype, int64_t rows, int width) {
  return dtype == BLOCK_F32 ? backward_bytes<F32>(rows, width) : backward_bytes<BF16>(rows, width);
}

}  // namespace block
