// Device-side building blocks of the layer's operators (gfx950, wave64):
// element types, activations with their derivatives, and the epilogues that
// every matrix kernel ends in.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

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
  static __device__ __forceinline__ uint32_t store2(float f, float g) {
    typedef __bf16 pair __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, pair{(__bf16)f, (__bf16)g});
  }
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
  static __device__ __forceinline__ uint32_t store2(float f, float g) {
    typedef _Float16 pair __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, pair{(_Float16)f, (_Float16)g});
  }
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

// sigmoid(z) from v_exp_f32 and v_rcp_f32 (1 ulp each; a full division would
// double the instructions of an epilogue that is bound by them).
__device__ __forceinline__ float sigmoid(float z) { return __builtin_amdgcn_rcpf(1.f + __expf(-z)); }

// GELU is z Phi(z), Phi the normal distribution's, and its slope Phi(z) +
// z exp(-z^2 / 2) / sqrt(2 pi). One exponential serves both: Phi(-|z|) =
// exp(-z^2 / 2) t Q(t), t = 1 / (1 + 0.3 |z|), where Q of degree 7 is a
// minimax fit (linear programme in the Chebyshev basis) of the relative error
// over 0 <= |z| <= 14.5; with the coefficients as they stand that error is
// 2.3e-7. Evaluated in FP32 the tail is off by 2.1e-7 absolute, and relative by
// 6e-7 up to |z| = 2, 2.2e-6 up to 6 and 8e-6 up to 13: the rounding of the
// exponential's argument, which grows with z^2. (1 + erf) / 2 would lose the
// negative tail altogether from -5.5 on.
// The ending of a tile whose CU has no other is bound by these instructions
// (200 rows of 1000 x 776 in whole tiles, with the slope kept: 25.1 us by the
// library's erff and one conversion per stored value, 19.6 like this).
// The tanh form of GELU is z sigmoid(2 y), y = sqrt(2/pi) (z + 0.044715 z^3).
// In derivatives the arguments of terms that vanish for large |z| are clamped
// where the term is already 0 in FP32, so that they stay 0 and not infinity
// times 0.
template <int Act>
__device__ __forceinline__ ValueSlope activate(float z) {
  if constexpr (Act == BLOCK_ACT_NONE) {
    return {z, 1.f};
  } else if constexpr (Act == BLOCK_ACT_RELU) {
    return {z < 0.f ? 0.f : z, z > 0.f ? 1.f : (z == z ? 0.f : z)};
  } else if constexpr (Act == BLOCK_ACT_SILU) {
    const float s = sigmoid(z);
    const float zc = fminf(fmaxf(z, -100.f), 100.f);  // s or 1 - s is 0 beyond 89
    return {z * s, s * (1.f + zc * (1.f - s))};
  } else if constexpr (Act == BLOCK_ACT_GELU) {
    const float x = fabsf(z), t = __builtin_amdgcn_rcpf(fmaf(0.3f, x, 1.f));
    float q = 0.0354313701f;
    q = fmaf(q, t, -0.156170219f);
    q = fmaf(q, t, 0.204543695f);
    q = fmaf(q, t, -0.0519903526f);
    q = fmaf(q, t, 0.127650067f);
    q = fmaf(q, t, 0.100195102f);
    q = fmaf(q, t, 0.120707922f);
    q = fmaf(q, t, 0.119632363f);
    const float e = __builtin_amdgcn_exp2f(z * z * -0.72134752044448170f);  // -log2(e) / 2
    const float tail = e * (t * q), cdf = z < 0.f ? tail : 1.f - tail;
    const float zc = fminf(fmaxf(z, -20.f), 20.f);  // e is 0 beyond 15
    return {z * cdf, cdf + zc * (e * 0.39894228040143268f)};
  } else {
    const float c = 1.5957691216057308f;  // 2 sqrt(2/pi)
    // exp(-2 y) with its factors joined with log2(e)
    const float s = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(z * fmaf(z * z, -0.10294324f, -2.3022082f)));
    const float zc = fminf(fmaxf(z, -10.f), 10.f);  // 1 - s is 0 or s is below 1e-37
    return {z * s, s + zc * s * (1.f - s) * c * (1.f + 3.f * 0.044715f * zc * zc)};
  }
}

// Calls f(activation constant): `act` is uniform over a launch, so this is one
// scalar branch around each whole use.
template <typename F>
__device__ __forceinline__ void with_activation(int act, F f) {
  switch (act) {
    case BLOCK_ACT_NONE: f(std::integral_constant<int, BLOCK_ACT_NONE>{}); break;
    case BLOCK_ACT_RELU: f(std::integral_constant<int, BLOCK_ACT_RELU>{}); break;
    case BLOCK_ACT_SILU: f(std::integral_constant<int, BLOCK_ACT_SILU>{}); break;
    case BLOCK_ACT_GELU: f(std::integral_constant<int, BLOCK_ACT_GELU>{}); break;
    default: f(std::integral_constant<int, BLOCK_ACT_GELU_TANH>{}); break;
  }
}

// --------------------------------------------------------------- epilogue --

// Up to C (4 or 8) consecutive columns of a row, `count` of them inside the
// matrix.
template <typename T, int C>
__device__ __forceinline__ void store_cols(typename T::raw* p, const float (&v)[C], int count) {
  uint32_t w[C / 2];
#pragma unroll
  for (int t = 0; t < C / 2; ++t) w[t] = T::store2(v[2 * t], v[2 * t + 1]);
  if (count >= C) {
    if constexpr (C == 8)
      reinterpret_cast<Any16*>(p)->v = u32x4{w[0], w[1], w[2], w[3]};
    else
      reinterpret_cast<Any8*>(p)->v = u32x2{w[0], w[1]};
    return;
  }
#pragma unroll
  for (int t = 0; t < C - 1; ++t)
    if (t < count) p[t] = (uint16_t)(w[t >> 1] >> (16 * (t & 1)));
}

template <typename T, int C>
__device__ __forceinline__ void load_cols(const typename T::raw* p, float (&v)[C], int count) {
  uint32_t w[C / 2] = {};
  if (count >= C) {
    if constexpr (C == 8) {
      const u32x4 x = reinterpret_cast<const Any16*>(p)->v;
      w[0] = x[0]; w[1] = x[1]; w[2] = x[2]; w[3] = x[3];
    } else {
      const u32x2 x = reinterpret_cast<const Any8*>(p)->v;
      w[0] = x[0]; w[1] = x[1];
    }
  } else {
#pragma unroll
    for (int t = 0; t < C - 1; ++t)
      if (t < count) w[t >> 1] |= (uint32_t)p[t] << (16 * (t & 1));
  }
#pragma unroll
  for (int t = 0; t < C; ++t) v[t] = T::load((uint16_t)(w[t >> 1] >> (16 * (t & 1))));
}

// The end of a product: `v` (and for the gated product `u`) are the FP32 sums
// of columns col .. col + C - 1 of output row `row`, `bias` and `residual`
// (kLinear; zeros if there is none) what is added before and after the
// activation; `which` selects the output matrix of a product with two.
// Everything happens in FP32 and each output is rounded once. Save: also the
// derivatives for the backward pass, rounded to the activations' type like
// everything else a training step keeps: FP32 would double the bytes of what
// is, per layer, the largest thing kept. It costs one rounding of three in
// the gradients (an RMS of 1.7 instead of 1.4 roundings).
template <typename T, int Mode, int Act, bool Save, int C>
__device__ __forceinline__ void finish(const GemmArgs& p, int which, int64_t row, int col, float (&v)[C],
                                       const float (&u)[C], const float (&bias)[C], const float (&residual)[C]) {
  typedef typename T::raw raw;
  const int count = p.n - col;
  if (row >= p.m || count <= 0) return;
  if constexpr (Mode == kGated || Mode == kLinear) {
    float d0[C], d1[C];
#pragma unroll
    for (int t = 0; t < C; ++t) {
      const ValueSlope s = activate<Act>(Mode == kLinear ? v[t] + bias[t] : v[t]);
      v[t] = Mode == kLinear ? s.a + residual[t] : s.a * u[t];
      d0[t] = Mode == kLinear ? s.d : s.d * u[t];
      d1[t] = s.a;
    }
    if constexpr (Save) {
      store_cols<T, C>(static_cast<raw*>(p.saved[0]) + row * p.n + col, d0, count);
      if (Mode == kGated) store_cols<T, C>(static_cast<raw*>(p.saved[1]) + row * p.n + col, d1, count);
    }
  }
  store_cols<T, C>(static_cast<raw*>(p.c[which]) + row * p.ldc + col, v, count);
}

// Calls f(activation constant, save constant) for the product `p` ends in.
template <int Mode, typename F>
__device__ __forceinline__ void with_ending(const GemmArgs& p, F f) {
  if constexpr (Mode == kGated || Mode == kLinear) {
    with_activation(p.act, [&](auto act) __attribute__((always_inline)) {
      if constexpr (Mode == kGated && decltype(act)::value == BLOCK_ACT_NONE) return;  // not a gated activation
      else if (decltype(act)::value != BLOCK_ACT_NONE && p.saved[0] != nullptr) f(act, std::true_type{});
      else f(act, std::false_type{});
    });
  } else {
    f(std::integral_constant<int, BLOCK_ACT_NONE>{}, std::false_type{});
  }
}

// finish() for one group of columns, bias and residual read here.
template <typename T, int Mode, int C>
__device__ __forceinline__ void epilogue(const GemmArgs& p, int which, int64_t row, int col, float (&v)[C],
                                         float (&u)[C]) {
  typedef typename T::raw raw;
  float bias[C] = {}, residual[C] = {};
  if (Mode == kLinear && row < p.m && col < p.n) {
    if (p.bias != nullptr) load_cols<T, C>(static_cast<const raw*>(p.bias) + col, bias, p.n - col);
    if (p.residual != nullptr)
      load_cols<T, C>(static_cast<const raw*>(p.residual) + row * p.ldr + col, residual, p.n - col);
  }
  with_ending<Mode>(p, [&](auto act, auto save) __attribute__((always_inline)) {
    finish<T, Mode, decltype(act)::value, decltype(save)::value, C>(p, which, row, col, v, u, bias, residual);
  });
}

}  // namespace block
