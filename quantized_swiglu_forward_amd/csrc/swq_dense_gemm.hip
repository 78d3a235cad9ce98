// Products with 16-bit weights: out[p, q] = act(sum_r a(p, r) b(q, r) + bias[q]) + res[p, q], each
// operand's inner index r along its rows or down its columns.
#include <algorithm>

#include "swq_dense.h"
#include "swq_dense_device.h"

namespace swq {
namespace {

template <int TYPE>
__device__ __forceinline__ f32x4 mfma_16(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (TYPE == kTypeF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                   0);
}

// 64 x 64 outputs per block, four waves of 32 x 32, 32 inner indexes at a time through LDS.
template <int TYPE>
__global__ __launch_bounds__(256) void dense_kernel(DenseGemm g) {
  constexpr int PITCH = 40;
  __shared__ __attribute__((aligned(16))) uint16_t la[64 * PITCH], lb[64 * PITCH];
  __shared__ float lz[64 * 65];
#ifdef SWQ_LDS_POISON
  lds_poison(la, sizeof(la), kPoisonFloat);
  lds_poison(lb, sizeof(lb), kPoisonFloat);
  lds_poison(lz, sizeof(lz), kPoisonFloat);
  __syncthreads();
#endif
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r16 = lane & 15, h = lane >> 4;
  const int64_t tq = (g.Q + 63) / 64;
  const int64_t p0 = (int64_t)blockIdx.x / tq * 64, q0 = (int64_t)blockIdx.x % tq * 64;
  const int wp = (wave >> 1) * 32, wq = (wave & 1) * 32;
  f32x4 acc[2][2] = {};
  const auto stage = [&](uint16_t* l, const uint16_t* x, int64_t ld, int way, int64_t i0, int64_t n, int64_t r0) {
    for (int e = tid; e < 64 * 32; e += 256) {
      const int i = way == kAlong ? e >> 5 : e & 63, r = way == kAlong ? e & 31 : e >> 6;
      const bool in = i0 + i < n && r0 + r < g.R;
      l[i * PITCH + r] = in ? x[way == kAlong ? (i0 + i) * ld + r0 + r : (r0 + r) * ld + i0 + i] : (uint16_t)0;
    }
  };
  for (int64_t r0 = 0; r0 < g.R; r0 += 32) {
    __syncthreads();
    stage(la, g.a, g.lda, g.way_a, p0, g.P, r0);
    stage(lb, g.b, g.ldb, g.way_b, q0, g.Q, r0);
    __syncthreads();
    u32x4 a[2], b[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      a[i] = *(const u32x4*)(la + (wp + 16 * i + r16) * PITCH + 8 * h);
      b[i] = *(const u32x4*)(lb + (wq + 16 * i + r16) * PITCH + 8 * h);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] = mfma_16<TYPE>(b[j], a[i], acc[i][j]);
  }
  // lane 16 h + r has columns 4 h .. 4 h + 3 of row r
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) lz[(wp + 16 * i + r16) * 65 + wq + 16 * j + 4 * h + e] = acc[i][j][e];
  __syncthreads();
  const int64_t blocks = (g.Q + 31) / 32;
  for (int e = tid; e < 64 * 64; e += 256) {          // a wave has a whole row
    const int i = e >> 6, j = e & 63;
    const int64_t p = p0 + i, q = q0 + j;
    const bool in = p < g.P && q < g.Q;
    float z = lz[i * 65 + j];
    if (in && g.bias) z += from_16(g.bias[q], TYPE);
    if (g.z_scales) {
      uint32_t m = in ? __float_as_uint(z) & 0x7FFFFFFFu : 0u;
#pragma unroll
      for (int d = 16; d; d >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d));
      const Mx8Step s = mx8_step(m);
      if (in) ((int8_t*)g.z)[p * g.Q + q] = (int8_t)mx8_code(z, s);
      if (in && (q & 31) == 0) g.z_scales[p * blocks + q / 32] = (uint8_t)s.byte;
    } else if (g.z && in) {
      ((uint16_t*)g.z)[p * g.Q + q] = to_16(z, TYPE);
    }
    if (!in) continue;
    float y = activate(z, g.act);
    if (g.res) y += from_16(g.res[p * g.Q + q], TYPE);
    if (g.out_type == kTypeF32) ((float*)g.out)[p * g.Q + q] = y;
    else ((uint16_t*)g.out)[p * g.Q + q] = to_16(y, TYPE);
  }
}

}  // namespace

hipError_t launch_dense_gemm(const DenseGemm& g, hipStream_t st) {
  const int64_t blocks = (g.P + 63) / 64 * ((g.Q + 63) / 64);
  if (blocks >= (int64_t(1) << 24)) return hipErrorInvalidValue;
  if (g.type == kTypeF16) dense_kernel<kTypeF16><<<(unsigned)blocks, 256, 0, st>>>(g);
  else dense_kernel<kTypeBf16><<<(unsigned)blocks, 256, 0, st>>>(g);
  return hipGetLastError();
}

}  // namespace swq
