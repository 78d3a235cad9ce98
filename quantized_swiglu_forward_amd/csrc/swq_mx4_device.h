// Device helpers of the microscaled 4-bit format (MXFP4): e2m1 codes, eight to
// a 32-bit word along K with code j in bits [4j, 4j+4), and one e8m0 scale byte
// b per 32 inputs, 2^(b - 127), 255 = NaN.
//
// The conversions are the target's own instructions.  Measured over every
// (scale byte, code) pair and over all bf16 inputs at scales from far below to
// far above the block's: decoding gives the exact product (byte 0 is 2^-127,
// byte 255 NaN, a value past float32's range infinity), encoding divides by
// the scale, rounds to nearest even and saturates at 6, for bf16, binary16
// and float32 inputs alike.  The scale operand is a float32 whose exponent
// field is the byte.
#pragma once

#include "swq_device.h"

// A lambda that is not inlined would take its captures, buffer descriptors among
// them, from memory.
#define SWQ_INLINE __attribute__((always_inline))

namespace swq {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ float e8m0_operand(uint32_t byte) { return __uint_as_float(byte << 23); }

// Eight codes of one word times 2^(byte - 127) as bf16 (exact: two significant bits).
__device__ __forceinline__ bf16x8 mx4_word(uint32_t w, float scale) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3);
  return (bf16x8){a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// Codes 2 E and 2 E + 1 of a word, likewise.
template <int E>
__device__ __forceinline__ uint32_t mx4_pair(uint32_t w, float scale) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, E));
}

// A binary16 value as the sum of two bf16 values: hi rounds it to 8
// significant bits, lo is the rest (at most 3 bits; both exact: bf16's
// exponent range holds binary16's).  An infinity or NaN is hi alone.
__device__ __forceinline__ void split_f16(_Float16 v, __bf16& hi, __bf16& lo) {
  const float f = (float)v;
  hi = (__bf16)f;
  const float rest = f - (float)hi;
  lo = (__bf16)(__builtin_isfinite(f) ? rest : 0.0f);
}

__device__ __forceinline__ void split_f16x8(f16x8 v, bf16x8& hi, bf16x8& lo) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    __bf16 a, b;
    split_f16(v[i], a, b);
    hi[i] = a;
    lo[i] = b;
  }
}

__device__ __forceinline__ f32x4 mfma_bf16(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// 128 codes of both operands, one block of 32 per lane: acc += sum a b 2^(sa + sb - 254).
__device__ __forceinline__ f32x4 mfma_mx4(u32x4 a, uint32_t sa, u32x4 b, uint32_t sb, f32x4 c) {
  const i32x8 A = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i32x8 B = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(A, B, c, 4, 4, 0, (int)sa, 0, (int)sb);
}

// What bf16 rounding leaves of a value, for a second bf16 operand (an infinity leaves nothing).
__device__ __forceinline__ float bf16_rest(float f) {
  const float hi = round_to_bf16(f);
  return __builtin_isfinite(hi) ? f - hi : 0.0f;
}

// 16-bit output types by number (0 bf16, 2 binary16).
__device__ __forceinline__ uint16_t to_16(float f, int type) { return type == 2 ? f32_to_f16(f) : f32_to_bf16(f); }
__device__ __forceinline__ float from_16(uint16_t b, int type) { return type == 2 ? f16_to_f32(b) : bf16_to_f32(b); }

template <int TYPE>
__device__ __forceinline__ uint32_t pack16(float a, float b) {
  return (uint32_t)to_16(a, TYPE) | (uint32_t)to_16(b, TYPE) << 16;
}

// Four consecutive outputs of one row, starting at column n of N.  `vec`: the
// row and the base allow one wide store.
__device__ __forceinline__ void store4(void* out, int64_t at, int n, int N, bool vec, f32x4 v, int type) {
  if (type == 1) {
    float* o = (float*)out + at + n;
    if (vec && n + 4 <= N) {
      *(f32x4*)o = v;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n + i < N) o[i] = v[i];
    }
    return;
  }
  uint16_t* o = (uint16_t*)out + at + n;
  uint16_t q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) q[i] = to_16(v[i], type);
  if (vec && n + 4 <= N) {
    *(u32x2*)o = (u32x2){(uint32_t)q[0] | (uint32_t)q[1] << 16, (uint32_t)q[2] | (uint32_t)q[3] << 16};
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < N) o[i] = q[i];
  }
}

}  // namespace swq
