// Device helpers of the products with 16-bit weights, the activations and
// their derivatives, and the 8-bit activation checkpoints.
#pragma once

#include "swq_dense.h"
#include "swq_mx4_device.h"

namespace swq {

typedef __attribute__((ext_vector_type(2), aligned(1))) uint32_t u32x2_any;   // at any address
typedef __attribute__((ext_vector_type(4), aligned(1))) uint32_t u32x4_any;

// i / n; 64-bit division is a long sequence of instructions.
__device__ __forceinline__ int64_t over(int64_t i, uint32_t n) {
  return (uint64_t)i >> 32 ? i / n : (int64_t)((uint32_t)i / n);
}

// ---- 8-bit checkpoints (MXINT8: int8 codes q, one e8m0 byte b per 32 neighbours of a row, q 2^(b - 133)) ----
//
// The step 2^e of a block is the smallest power of two, from 2^-126 on, at which no element's
// code passes 127: amax lies in [64, 128) steps, or in [127.5, 128) the step is the next one.
// Codes of 7 bits times a power of two are exact in bf16 (and in binary16 down to its own grid, which the
// values of binary16 inputs lie on): the one rounding is the code's, at most half a step, that is amax / 127 from
// amax = 2^-120 on (next to float32's largest value, where the step can be no larger, a whole one).
// A block with an infinity or a NaN gets byte 255 (NaN) and zero codes.

struct Mx8Step {
  float inverse;            // 2^-e
  uint32_t byte;
};
__device__ __forceinline__ Mx8Step mx8_step(uint32_t amax_bits) {
  const int field = (int)(amax_bits >> 23);
  if (field == 255) return {0.0f, 255u};
  int e = max(field - 133, -126);
  const float top = __uint_as_float(amax_bits) * __uint_as_float((uint32_t)(127 - e) << 23);
  if (top >= 127.5f && e < 121) ++e;           // (2^121 is the last: byte 255 says NaN)
  return {__uint_as_float((uint32_t)(127 - e) << 23), (uint32_t)(e + 133)};
}

// The largest magnitude's bits of eight values (a NaN's are the largest).
__device__ __forceinline__ uint32_t mx8_amax(const float (&v)[8]) {
  float m = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = __builtin_elementwise_maximum(fabsf(v[j]), m);
  return __float_as_uint(m) & 0x7FFFFFFFu;
}

// Eight codes.  Adding 1.5 2^23 rounds a value below 2^22 to a whole number, ties to even, and leaves it in the low
// bits.  Only next to float32's largest value can that be 128, and only a NaN block (byte 255) holds values that are no
// numbers: both go the long way.
__device__ __forceinline__ u32x2 mx8_codes(const float (&v)[8], Mx8Step s) {
  uint32_t q[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) q[j] = __float_as_uint(fmaf(v[j], s.inverse, 12582912.0f));
  if (__any(s.byte >= 254)) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float r = __builtin_amdgcn_fmed3f(rintf(v[j] * s.inverse), -127.0f, 127.0f);
      q[j] = s.byte == 255 ? 0u : (uint32_t)(int)r;
    }
  }
  u32x2 w;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t lo = __builtin_amdgcn_perm(q[4 * i + 1], q[4 * i], 0x0C0C0400u);
    const uint32_t hi = __builtin_amdgcn_perm(q[4 * i + 3], q[4 * i + 2], 0x04000C0Cu);
    w[i] = lo | hi;
  }
  return w;
}

// 2^(b - 133) (bytes below 7, which the quantiser never writes: subnormal), NaN for 255
__device__ __forceinline__ float mx8_scale(uint32_t byte) {
  if (byte == 255) return __uint_as_float(0x7FC00000u);
  return __uint_as_float(byte > 6 ? (byte - 6) << 23 : 0x400000u >> (6 - byte));
}
__device__ __forceinline__ float mx8_value(uint32_t word, int i, float scale) {
  return (float)(int8_t)(word >> (8 * i)) * scale;
}

// ---- activations --------------------------------------------------------------------------------------------
//
// sigma(t) = 1 / (1 + 2^(-t log2 e)) from the hardware exp2 and reciprocal (about 1 ulp each).
__device__ __forceinline__ float sigma(float t) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(t * -1.4426950408889634f));
}

// The normal distribution's tail above |t|, 1 - Phi(|t|), and its density's e^(-t^2 / 2): Abramowitz and Stegun,
// Handbook of Mathematical Functions, 7.1.26 (erfc x = (a1 u + ... + a5 u^5) e^(-x^2), u = 1 / (1 + p x), absolute error below 1.5e-7)
// at x = |t| / sqrt 2.
__device__ __forceinline__ float normal_tail(float t, float& e) {
  const float x = fabsf(t) * 0.70710678118654752f;
  const float u = __builtin_amdgcn_rcpf(fmaf(0.3275911f, x, 1.0f));
  e = __builtin_amdgcn_exp2f(t * t * -0.72134752044448170f);
  float s = fmaf(u, 1.061405429f, -1.453152027f);
  s = fmaf(u, s, 1.421413741f);
  s = fmaf(u, s, -0.284496736f);
  s = fmaf(u, s, 0.254829592f);
  return 0.5f * s * u * e;
}

// (1 + tanh(sqrt(2 / pi) (t + 0.044715 t^3))) / 2 = sigma(2 sqrt(2 / pi) (t + 0.044715 t^3))
__device__ __forceinline__ float gelu_sigma(float t) {
  return sigma(1.5957691216057308f * fmaf(0.044715f * t * t, t, t));
}

__device__ __forceinline__ float activate(float z, int act) {
  if (act == kActNone) return z;
  if (act == kActRelu) return z > 0.0f ? z : z != z ? z : 0.0f;
  if (act == kActSilu) return z * sigma(z);
  if (act == kActGelu) {
    float e;
    const float tail = normal_tail(z, e);
    return z * (z < 0.0f ? tail : 1.0f - tail);
  }
  return z * gelu_sigma(z);
}

// d activate / dz (relu: 0 at 0).  Where an intermediate square overflows, the exponential that multiplies it is 0
// and the derivative its limit.  An infinite z (a kept z past its 16-bit type's largest value is one) is a factor of float32's
// largest value instead, as the other factor is 0 there; of a NaN the other factor is one too.
__device__ __forceinline__ float as_factor(float z) {
  constexpr float top = 3.402823466e38f;
  return __builtin_amdgcn_fmed3f(z, -top, top);
}
__device__ __forceinline__ float activate_slope(float z, int act) {
  if (act == kActNone) return 1.0f;
  if (act == kActRelu) return z > 0.0f ? 1.0f : z != z ? z : 0.0f;
  if (act == kActSilu) {
    const float s = sigma(z);
    return s * fmaf(as_factor(z), 1.0f - s, 1.0f);
  }
  if (act == kActGelu) {
    float e;
    const float tail = normal_tail(z, e);
    return fmaf(as_factor(z) * e, 0.39894228040143268f, z < 0.0f ? tail : 1.0f - tail);
  }
  const float s = gelu_sigma(z), d = s * (1.0f - s);
  return d > 0.0f ? fmaf(z * d, 1.5957691216057308f * fmaf(3.0f * 0.044715f * z, z, 1.0f), s) : s;
}

}  // namespace swq
