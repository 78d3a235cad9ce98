// MXFP4 quantisation and its inverse.
//
// A block of 32 inputs has the scale 2^e with e = floor(log2 max|x|) - 2
// clamped to [-127, 127] (2 is e2m1's largest exponent; an all-zero block takes
// -127), so the block's largest element divided by it lies in [4, 8) and
// saturates at 6.  An infinity or NaN makes the block's scale NaN (byte
// 255) with codes 0.
#include "swq_mx4.h"
#include "swq_mx4_device.h"

namespace swq {
namespace {

// Bound by the bytes: 8192 x 10240 bf16 (168 MB in, 45 MB out) takes 43 us, 5.0 TB/s (a
// large copy reaches 5.2); its inverse 31 us, the codes still in the last-level
// cache.  48 x 2048 takes 2.5 us each, one load's latency and the launch.

// One thread per 8 inputs (one word of codes), four threads per block: a wave reads one contiguous
// kilobyte (16-bit inputs) and writes 256 bytes, and the block's maximum is two
// lane exchanges.  Maximum and scale are exact; the one rounding is the code's.
template <int TYPE>
__global__ __launch_bounds__(256) void mx4_quantize_kernel(const void* __restrict__ x, int64_t words,
                                                           uint32_t* __restrict__ codes,
                                                           uint8_t* __restrict__ scales) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= words) return;                      // words is a multiple of 4: whole blocks leave together
  float v[8];
  if constexpr (TYPE == kTypeF32) {
    const f32x4 a = ((const f32x4*)x)[2 * i], b = ((const f32x4*)x)[2 * i + 1];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = a[j], v[4 + j] = b[j];
  } else {
    const u32x4 a = ((const u32x4*)x)[i];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = from_16((uint16_t)(a[j >> 1] >> (16 * (j & 1))), TYPE);
  }
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7FFFFFFFu);
  m = max(m, (uint32_t)__shfl_xor((int)m, 1));
  m = max(m, (uint32_t)__shfl_xor((int)m, 2));
  const uint32_t field = m >> 23;              // 0 for zero and float32's subnormals: byte 0 either way
  uint32_t byte = field > 2 ? field - 2 : 0, w = 0;
  if (field == 255) {
    byte = 255;
  } else {
    const float sc = e8m0_operand(byte);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], sc, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], sc, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], sc, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], sc, 3);
  }
  codes[i] = w;
  if ((i & 3) == 0) scales[i >> 2] = (uint8_t)byte;
}

// One thread per word of codes.  code * 2^e is exact in float32 and rounded once, to nearest even, for
// 16-bit outputs.
template <int TYPE>
__global__ __launch_bounds__(256) void mx4_dequantize_kernel(const uint32_t* __restrict__ codes,
                                                             const uint8_t* __restrict__ scales, int64_t words,
                                                             void* __restrict__ out) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= words) return;
  const uint32_t w = codes[i];
  const float sc = e8m0_operand(scales[i >> 2]);
  const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, sc, 0);
  const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, sc, 1);
  const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, sc, 2);
  const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, sc, 3);
  if constexpr (TYPE == kTypeF32) {
    ((f32x4*)out)[2 * i] = (f32x4){a[0], a[1], b[0], b[1]};
    ((f32x4*)out)[2 * i + 1] = (f32x4){c[0], c[1], d[0], d[1]};
  } else {
    const auto pk = [](f32x2 v) { return (uint32_t)to_16(v[0], TYPE) | (uint32_t)to_16(v[1], TYPE) << 16; };
    ((u32x4*)out)[i] = (u32x4){pk(a), pk(b), pk(c), pk(d)};
  }
}

// One launch holds fewer than 2^32 threads (of more the rest is left out, with no error); words past
// kLaunchWords go to further launches.
constexpr int64_t kLaunchWords = int64_t(1) << 30;

template <int TYPE>
void quantize_as(const void* x, int64_t words, uint32_t* codes, uint8_t* scales, hipStream_t st) {
  for (int64_t w = 0; w < words; w += kLaunchWords) {
    const int64_t n = words - w < kLaunchWords ? words - w : kLaunchWords;
    mx4_quantize_kernel<TYPE><<<dim3((unsigned)((n + 255) / 256)), 256, 0, st>>>(
        (const char*)x + w * 8 * type_bytes(TYPE), n, codes + w, scales + w / 4);
  }
}

template <int TYPE>
void dequantize_as(const uint32_t* codes, const uint8_t* scales, int64_t words, void* out, hipStream_t st) {
  for (int64_t w = 0; w < words; w += kLaunchWords) {
    const int64_t n = words - w < kLaunchWords ? words - w : kLaunchWords;
    mx4_dequantize_kernel<TYPE><<<dim3((unsigned)((n + 255) / 256)), 256, 0, st>>>(
        codes + w, scales + w / 4, n, (char*)out + w * 8 * type_bytes(TYPE));
  }
}

}  // namespace

hipError_t launch_mx4_quantize(const void* x, int64_t blocks, int type, uint32_t* codes, uint8_t* scales,
                               hipStream_t st) {
  const int64_t words = blocks * 4;
  if (type == kTypeF32) quantize_as<kTypeF32>(x, words, codes, scales, st);
  else if (type == kTypeF16) quantize_as<kTypeF16>(x, words, codes, scales, st);
  else quantize_as<kTypeBf16>(x, words, codes, scales, st);
  return hipGetLastError();
}

hipError_t launch_mx4_dequantize(const uint32_t* codes, const uint8_t* scales, int64_t blocks, int type, void* out,
                                 hipStream_t st) {
  const int64_t words = blocks * 4;
  if (type == kTypeF32) dequantize_as<kTypeF32>(codes, scales, words, out, st);
  else if (type == kTypeF16) dequantize_as<kTypeF16>(codes, scales, words, out, st);
  else dequantize_as<kTypeBf16>(codes, scales, words, out, st);
  return hipGetLastError();
}

}  // namespace swq
