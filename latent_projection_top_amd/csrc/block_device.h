// Device-side building blocks of the layer's operators (gfx950, wave64):
// element types, activations with their derivatives, and the epilogues that
// every matrix kernel ends in.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "block_launch.h"

namespace block {

constexpr int kWave = 64;

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
// 16 bytes at any element-aligned address: one dwordx4 load or store on
// gfx950, whose global memory accesses need no alignment beyond their element
// type's.
struct __attribute__((packed, aligned(2))) Any16 { u32x4 v; };
struct __attribute__((packed, aligned(2))) Any8 { u32x2 v; };

// ---------------------------------------------------------- element types --

struct BF16 {
  typedef uint16_t raw;
  typedef __bf16 frag __attribute__((ext_vector_type(8)));
  static constexpr int code = BLOCK_BF16;
  static __device__ __forceinline__ float load(raw r) { return __uint_as_float((uint32_t)r << 16); }
  // nearest-even, NaN stays NaN (v_cvt_pk_bf16_f32)
  static __device__ __forceinline__ raw store(float f) { return __builtin_bit_cast(raw, (__bf16)f); }
  static __device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(frag, a), __builtin_bit_cast(frag, b),
                                                  c, 0, 0, 0);
  }
};

struct F16 {
  typedef uint16_t raw;
  typedef _Float16 frag __attribute__((ext_vector_type(8)));
  static constexpr int code = BLOCK_F16;
  static __device__ __forceinline__ float load(raw r) { return (float)__builtin_bit_cast(_Float16, r); }
  static __device__ __forceinline__ raw store(float f) { return __builtin_bit_cast(raw, (_Float16)f); }
  static __device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(frag, a), __builtin_bit_cast(frag, b),
                                                 c, 0, 0, 0);
  }
};

struct F32 {
  typedef float raw;
  static constexpr int code = BLOCK_F32;
  static __device__ __forceinline__ float load(raw r) { return r; }
  static __device__ __forceinline__ raw store(float f) { return f; }
};

// A value of runtime type `dtype` (the norm's parameters).
__device__ __forceinline__ float load_param(const void* p, int64_t i, int dtype) {
  if (dtype == BLOCK_F32) return static_cast<const float*>(p)[i];
  const uint16_t r = static_cast<const uint16_t*>(p)[i];
  return dtype == BLOCK_BF16 ? BF16::load(r) : F16::load(r);
}

__device__ __forceinline__ void store_param(void* p, int64_t i, int dtype, float v) {
  if (dtype == BLOCK_F32)
    static_cast<float*>(p)[i] = v;
  else
    static_cast<uint16_t*>(p)[i] = dtype == BLOCK_BF16 ? BF16::store(v) : F16::store(v);
}

// ------------------------------------------------------------ activations --

struct ValueSlope {
  float a;  // act(z)
  float d;  // act'(z)
};

// `act` is uniform over a launch, so the switch is one scalar branch. The
// arguments of terms that vanish for large |z| are clamped where the term is
// already 0 in FP32, so that they stay 0 and not infinity times 0.
__device__ __forceinline__ ValueSlope activate(int act, float z) {
  switch (act) {
    case BLOCK_ACT_RELU:
      return {z < 0.f ? 0.f : z, z > 0.f ? 1.f : (z == z ? 0.f : z)};
    case BLOCK_ACT_SILU: {
      const float s = 1.f / (1.f + __expf(-z));
      return {z * s, s * (1.f + z * (1.f - s))};
    }
    case BLOCK_ACT_GELU: {
      const float cdf = 0.5f * (1.f + erff(z * 0.70710678118654752f));
      const float zc = fminf(fmaxf(z, -20.f), 20.f);  // exp(-200) is 0 in FP32
      return {z * cdf, cdf + zc * (__expf(-0.5f * zc * zc) * 0.39894228040143268f)};
    }
    case BLOCK_ACT_GELU_TANH: {
      const float c = 0.79788456080286536f;
      const float zc = fminf(fmaxf(z, -10.f), 10.f);  // tanh of +-43 is +-1 in FP32
      const float q = zc * zc;
      const float t = 1.f - 2.f / (1.f + __expf(2.f * c * zc * (1.f + 0.044715f * q)));
      const float half = 0.5f * (1.f + t);
      return {z * half, half + 0.5f * zc * (1.f - t * t) * c * (1.f + 3.f * 0.044715f * q)};
    }
    default:
      return {z, 1.f};
  }
}

// --------------------------------------------------------------- epilogue --

// Store up to four consecutive columns of a row (`count` of them, 4 unless
// the matrix ends inside).
template <typename T>
__device__ __forceinline__ void store4(typename T::raw* p, f32x4 v, int count) {
  if (count == 4) {
    const u32x2 w = {(uint32_t)T::store(v[0]) | (uint32_t)T::store(v[1]) << 16,
                     (uint32_t)T::store(v[2]) | (uint32_t)T::store(v[3]) << 16};
    reinterpret_cast<Any8*>(p)->v = w;
    return;
  }
#pragma unroll
  for (int t = 0; t < 3; ++t)
    if (t < count) p[t] = T::store(v[t]);
}

template <typename T>
__device__ __forceinline__ f32x4 load4(const typename T::raw* p, int count) {
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  if (count == 4) {
    const u32x2 w = reinterpret_cast<const Any8*>(p)->v;
#pragma unroll
    for (int t = 0; t < 4; ++t) v[t] = T::load((uint16_t)(w[t >> 1] >> (16 * (t & 1))));
    return v;
  }
#pragma unroll
  for (int t = 0; t < 3; ++t)
    if (t < count) v[t] = T::load(p[t]);
  return v;
}

// The end of a product: `v` (and for the gated product `u`) are the FP32 sums
// of columns col .. col + 3 of output row `row`; `which` selects the output
// matrix of a product with two. Everything happens in FP32 and each output is
// rounded once.
template <typename T, int Mode>
__device__ __forceinline__ void epilogue(const GemmArgs& p, int which, int64_t row, int col, f32x4 v,
                                         f32x4 u) {
  typedef typename T::raw raw;
  const int count = min(4, p.n - col);
  if (row >= p.m || count <= 0) return;
  raw* c = static_cast<raw*>(p.c[which]) + row * p.ldc + col;
  if constexpr (Mode == kGated) {
    f32x4 h, dg, du;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const ValueSlope s = activate(p.act, v[t]);
      h[t] = s.a * u[t];
      dg[t] = s.d * u[t];
      du[t] = s.a;
    }
    store4<T>(c, h, count);
    if (p.saved[0] != nullptr) {
      store4<T>(static_cast<raw*>(p.saved[0]) + row * p.n + col, dg, count);
      store4<T>(static_cast<raw*>(p.saved[1]) + row * p.n + col, du, count);
    }
  } else if constexpr (Mode == kLinear) {
    if (p.bias != nullptr) v += load4<T>(static_cast<const raw*>(p.bias) + col, count);
    if (p.act != BLOCK_ACT_NONE) {
      f32x4 d;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const ValueSlope s = activate(p.act, v[t]);
        v[t] = s.a;
        d[t] = s.d;
      }
      if (p.saved[0] != nullptr) store4<T>(static_cast<raw*>(p.saved[0]) + row * p.n + col, d, count);
    }
    if (p.residual != nullptr)
      v += load4<T>(static_cast<const raw*>(p.residual) + row * p.ldr + col, count);
    store4<T>(c, v, count);
  } else {
    store4<T>(c, v, count);
  }
}

}  // namespace block
