// Values as 8-bit integers with a common scale.
#pragma once

#include "experts_device.h"

namespace experts {

// The integers of values whose largest magnitude is `most`: q = rne(127 x / a),
// s = a / 127. The quotient is decided without a division: with x and a of at
// most 11 significant bits it is a border n + 1/2 exactly or at least 2^-19 of
// its size from one, and t below, a product corrected by its exact residual
// (fma), is within an ulp of it and equal where it is representable, as every
// border is. Values so small that 1 / a overflows, or so large that 127 x does,
// are scaled first, exactly.
struct Quantiser {
  float up, inv, a, s;
  Quantiser() = default;
  __device__ __forceinline__ explicit Quantiser(float most) {
    const float shift = most < 0x1p-60f ? 0x1p+100f : most > 0x1p+60f ? 0x1p-100f : 1.f;
    a = most * shift;
    up = 127.f * shift;
    inv = a > 0.f ? 1.f / a : 0.f;
    s = most / 127.f;
    if (!(most < INFINITY)) {  // infinite or NaN: the whole row is NaN
      a = inv = up = 0.f;
      s = NAN;
    }
  }
  // The integer in the low byte; adding 1.5 x 2^23 rounds to nearest-even. (Any
  // byte will do where the scale is NaN.)
  __device__ __forceinline__ uint32_t byte(float x) const {
    const float n = up * x, t = n * inv;
    return __float_as_uint(fmaf(fmaf(-t, a, n), inv, t) + 12582912.f);
  }
  __device__ __forceinline__ uint32_t bytes(float x, float y, float z, float w) const {
    const uint32_t lo = __builtin_amdgcn_perm(byte(y), byte(x), 0x0c0c0400);
    const uint32_t hi = __builtin_amdgcn_perm(byte(w), byte(z), 0x0c0c0400);
    return lo | hi << 16;
  }
  // sixteen values of a type, as they are in memory
  template <typename T>
  __device__ __forceinline__ u32x4 sixteen(u32x4 x, u32x4 y) const {
    u32x4 b;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const u32x4 v = e < 2 ? x : y;
      const uint32_t lo = v[2 * (e & 1)], hi = v[2 * (e & 1) + 1];
      b[e] = bytes(T::load((uint16_t)lo), T::load((uint16_t)(lo >> 16)), T::load((uint16_t)hi),
                   T::load((uint16_t)(hi >> 16)));
    }
    return b;
  }
};

// Largest magnitude of a type's values as the bits of one of them, which are in
// order for what has no sign: infinity and NaN come last.
template <typename T>
__device__ __forceinline__ float magnitude(uint32_t bits) {
  return T::load((uint16_t)bits);
}

// The larger magnitudes, two at a time, of what there is and eight values more.
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ u16x2 larger(u16x2 m, u32x4 v) {
#pragma unroll
  for (int e = 0; e < 4; ++e)
    m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, v[e] & 0x7fff7fffu));
  return m;
}

}  // namespace experts
