// 8-bit activation checkpoints, the SwiGLU that leaves them behind and its
// gradient, and the gradient of a product's activation with the bias's sums.
#include <algorithm>

#include "swq_dense.h"
#include "swq_dense_device.h"

namespace swq {
namespace {

// A tensor [R, K] in pieces of eight neighbours of a row, four pieces to a block of 32 (the last of a row may be
// shorter, and its pieces empty).  Piece i is piece i % (4 blocks) of row i / (4 blocks).
struct Pieces {
  int64_t R, K;
  uint32_t per_row;         // 4 ceil(K / 32)
};
struct Piece {
  int64_t at;               // its first element
  int64_t block;            // its block's scale
  int n;                    // elements, 0 .. 8
};
__device__ __forceinline__ Piece piece_of(const Pieces& t, int64_t i) {
  const int64_t row = over(i, t.per_row);
  const uint32_t c = (uint32_t)(i - row * t.per_row);
  const int64_t left = t.K - 8 * (int64_t)c;
  return {row * t.K + 8 * (int64_t)c, row * (t.per_row / 4) + (c >> 2), left >= 8 ? 8 : left > 0 ? (int)left : 0};
}

template <int TYPE>
__device__ __forceinline__ void load8(const void* x, int64_t at, int n, float* v) {
  if constexpr (TYPE == kTypeF32) {
    const uint32_t* f = (const uint32_t*)x + at;
    if (n == 8) {
      const u32x4 a = *(const u32x4_any*)f, b = *(const u32x4_any*)(f + 4);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = __uint_as_float(a[j]), v[4 + j] = __uint_as_float(b[j]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = j < n ? __uint_as_float(f[j]) : 0.0f;
    }
  } else {
    const uint16_t* f = (const uint16_t*)x + at;
    if (n == 8) {
      const u32x4 a = *(const u32x4_any*)f;
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = from_16((uint16_t)(a[j >> 1] >> (16 * (j & 1))), TYPE);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = j < n ? from_16(f[j], TYPE) : 0.0f;
    }
  }
}

template <int TYPE>
__device__ __forceinline__ void store8(void* y, int64_t at, int n, const float* v) {
  if constexpr (TYPE == kTypeF32) {
    float* f = (float*)y + at;
    if (n == 8) {
      *(u32x4_any*)f = __builtin_bit_cast(u32x4, (f32x4){v[0], v[1], v[2], v[3]});
      *(u32x4_any*)(f + 4) = __builtin_bit_cast(u32x4, (f32x4){v[4], v[5], v[6], v[7]});
    } else {
      for (int j = 0; j < n; ++j) f[j] = v[j];
    }
  } else {
    uint16_t* f = (uint16_t*)y + at;
    if (n == 8) {
      *(u32x4_any*)f = (u32x4){pack16<TYPE>(v[0], v[1]), pack16<TYPE>(v[2], v[3]), pack16<TYPE>(v[4], v[5]),
                               pack16<TYPE>(v[6], v[7])};
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < n) f[j] = to_16(v[j], TYPE);
    }
  }
}

__device__ __forceinline__ void decode8(const void* codes, float scale, int64_t at, int n, float* v) {
  const uint8_t* c = (const uint8_t*)codes + at;
  u32x2 w = {0u, 0u};
  if (n == 8) {
    w = *(const u32x2_any*)c;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) w[j >> 2] |= (uint32_t)c[j] << (8 * (j & 3));
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = mx8_value(w[j >> 2], j & 3, scale);
}

// Values of a checkpoint as TYPE: what rounds past binary16's largest value (a code's half step above it) is that value.
template <int TYPE>
__device__ __forceinline__ void hold8(float (&v)[8]) {
  if constexpr (TYPE == kTypeF16) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = v[j] != v[j] ? v[j] : __builtin_amdgcn_fmed3f(v[j], -65504.0f, 65504.0f);
  }
}

// The block's maximum over its four pieces (neighbouring lanes), codes and scale.
__device__ __forceinline__ void encode8(const float (&v)[8], const Piece& p, void* codes, uint8_t* scales) {
  uint32_t m = mx8_amax(v);
  m = max(m, (uint32_t)__shfl_xor((int)m, 1));
  m = max(m, (uint32_t)__shfl_xor((int)m, 2));
  const Mx8Step s = mx8_step(m);
  const u32x2 w = mx8_codes(v, s);
  uint8_t* c = (uint8_t*)codes + p.at;
  if (p.n == 8) {
    *(u32x2_any*)c = w;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < p.n) c[j] = (uint8_t)(w[j >> 2] >> (8 * (j & 3)));
  }
  if ((threadIdx.x & 3) == 0) scales[p.block] = (uint8_t)s.byte;
}

// The elementwise kernels: eight neighbours to a thread, so that every tensor moves in 16-byte pieces (codes in 8), a
// block's maximum is two exchanges between lanes, and nothing is read twice.  Memory bounds them: 8192 x 10240 bf16
// quantised in 47 us and back in 38 (5.4 and 6.7 TB/s, codes and a part of the values still in the last-level cache; of
// other tensors 45); the SwiGLU of 2048 x 14336 with both checkpoints 41 to 48 (237 MB), its gradient with the hidden tensor 51
// to 55 (295 MB).  Rows of odd lengths, 16 bytes at odd elements: 8192 x 10241 49 and 50, 2048 x 14337 46 and 57, so 4 to 11 %
// longer.  Small tensors take a launch's 2.5 to 3 us.
template <int TYPE>
__global__ __launch_bounds__(256) void mx8_quantize_kernel(const void* __restrict__ x, Pieces t, int64_t first,
                                                           int64_t end, void* __restrict__ codes,
                                                           uint8_t* __restrict__ scales) {
  const int64_t i = first + (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= end) return;                        // whole blocks leave together
  const Piece p = piece_of(t, i);
  float v[8];
  load8<TYPE>(x, p.at, p.n, v);
  encode8(v, p, codes, scales);
}

template <int TYPE>
__global__ __launch_bounds__(256) void mx8_dequantize_kernel(const void* __restrict__ codes,
                                                             const uint8_t* __restrict__ scales, Pieces t,
                                                             int64_t first, int64_t end, void* __restrict__ out) {
  const int64_t i = first + (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= end) return;
  const Piece p = piece_of(t, i);
  float v[8];
  decode8(codes, mx8_scale(scales[p.block]), p.at, p.n, v);
  hold8<TYPE>(v);
  store8<TYPE>(out, p.at, p.n, v);
}

template <int TYPE>
__global__ __launch_bounds__(256) void swiglu_kernel(const uint16_t* __restrict__ gate,
                                                     const uint16_t* __restrict__ up, Pieces t, int64_t first,
                                                     int64_t end, uint16_t* __restrict__ hidden,
                                                     void* __restrict__ gcodes, uint8_t* __restrict__ gscales,
                                                     void* __restrict__ ucodes, uint8_t* __restrict__ uscales) {
  const int64_t i = first + (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= end) return;
  const Piece p = piece_of(t, i);
  float g[8], u[8], y[8];
  load8<TYPE>(gate, p.at, p.n, g);
  load8<TYPE>(up, p.at, p.n, u);
#pragma unroll
  for (int j = 0; j < 8; ++j) y[j] = silu_times(g[j], u[j]);
  store8<TYPE>(hidden, p.at, p.n, y);
  if (gcodes) {
    encode8(g, p, gcodes, gscales);
    encode8(u, p, ucodes, uscales);
  }
}

template <int TYPE>
__device__ __forceinline__ void load_kept(const Kept& x, const Piece& p, float* v) {
  if (x.scales) decode8(x.data, mx8_scale(x.scales[p.block]), p.at, p.n, v);
  else load8<TYPE>(x.data, p.at, p.n, v);
}

template <int TYPE>
__global__ __launch_bounds__(256) void swiglu_backward_kernel(const uint16_t* __restrict__ dhidden, Kept gate, Kept up,
                                                              Pieces t, int64_t first, int64_t end,
                                                              uint16_t* __restrict__ dgate, uint16_t* __restrict__ dup,
                                                              uint16_t* __restrict__ hidden) {
  const int64_t i = first + (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= end) return;
  const Piece p = piece_of(t, i);
  float d[8], g[8], u[8], y[8];
  load8<TYPE>(dhidden, p.at, p.n, d);
  load_kept<TYPE>(gate, p, g);
  load_kept<TYPE>(up, p, u);
  if (hidden) {
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = silu_times(g[j], u[j]);
    store8<TYPE>(hidden, p.at, p.n, y);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float s = sigma(g[j]);
    u[j] = d[j] * u[j] * (s * fmaf(g[j], 1.0f - s, 1.0f));
    y[j] = d[j] * (g[j] * s);
  }
  store8<TYPE>(dgate, p.at, p.n, u);
  store8<TYPE>(dup, p.at, p.n, y);
}

// One launch holds fewer than 2^32 threads (of more the rest is left out, with no error).
constexpr int64_t kLaunchPieces = int64_t(1) << 30;

template <class F>
hipError_t over_pieces(int64_t R, int64_t K, F launch) {
  const Pieces t{R, K, (uint32_t)((K + 31) / 32 * 4)};
  const int64_t all = R * t.per_row;
  for (int64_t i = 0; i < all; i += kLaunchPieces) {
    const int64_t end = std::min(all, i + kLaunchPieces);
    launch(dim3((unsigned)((end - i + 255) / 256)), t, i, end);
  }
  return hipGetLastError();
}

// dz and the sums of its columns.  A block has a stretch of rows of 8 L columns (512; of narrow tensors the power of two
// that holds a row), eight of a row to a thread, 256 / L rows at a time; these meet in LDS, the stretches' sums in a
// later kernel, all in order.  One pass over dout and z is all there is to do, so memory bounds it: with x's checkpoint decoded by
// other blocks of the launch, 2048 x 4096 x 14336 takes 33 to 37 us (4.7 TB/s); the sums alone 25 to 27, of 14337 columns 31 to 35.
//
// dz is rounded to the operands' 16 bits here, once: that is what the matrix units take, and the precision that a layer's
// gradient has wherever it is kept as a tensor.  dx and dW are off by 0.0023 (bf16) and 0.00029 (binary16) in norm for it, 0.0017
// and 0.00021 with a float32 dz, which would need two products (a high and a low part) in place of each.  The bias's sums take dz
// before the rounding.  Past binary16's largest value dz is an infinity, as any gradient that needs a smaller loss scale.
template <int TYPE>
__device__ __forceinline__ void act_backward(const Prep& p, int64_t column_block, int64_t stretch, int64_t rows, int L,
                                             float* meet) {
  const Kept& z = p.z;
  const int64_t M = p.M, N = p.N;
  const int c = threadIdx.x & (L - 1), team = threadIdx.x / L, teams = 256 / L;
  const int64_t q = column_block * 8 * L + 8 * c, blocks = (N + 31) / 32, ld = (N + 7) / 8 * 8;
  const int n = q + 8 <= N ? 8 : q < N ? (int)(N - q) : 0;
  const int64_t m1 = min((stretch + 1) * rows, M);
  float sum[8] = {};
  const auto go = [&](auto slope) SWQ_INLINE {
    if (n > 0) {
#pragma unroll 2
      for (int64_t m = stretch * rows + team; m < m1; m += teams) {
        float d[8], v[8] = {};
        load8<TYPE>(p.dout, m * N + q, n, d);
        if (p.act != kActNone) {
          if (z.scales) decode8(z.data, mx8_scale(z.scales[m * blocks + q / 32]), m * N + q, n, v);
          else load8<TYPE>(z.data, m * N + q, n, v);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          d[j] = j < n ? d[j] * slope(v[j]) : 0.0f;
          sum[j] += d[j];
        }
        if (p.dz) store8<TYPE>(p.dz, m * ld + q, 8, d);      // (zeros behind a row's end)
      }
    }
  };
  switch (p.act) {
    case kActNone: go([](float) { return 1.0f; }); break;
    case kActRelu: go([](float v) { return activate_slope(v, kActRelu); }); break;
    case kActSilu: go([](float v) { return activate_slope(v, kActSilu); }); break;
    case kActGelu: go([](float v) { return activate_slope(v, kActGelu); }); break;
    default: go([](float v) { return activate_slope(v, kActGeluTanh); });
  }
  if (!p.sums && !p.dbias) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) meet[(team * L + c) * 8 + j] = sum[j];
  __syncthreads();
  for (int t = threadIdx.x; t < 8 * L; t += 256) {
    const int64_t column = column_block * 8 * L + t;
    if (column >= N) continue;
    float all = 0.0f;
#pragma unroll 4
    for (int i = 0; i < teams; ++i) all += meet[i * L * 8 + t];
    if (p.dbias) p.dbias[column] = to_16(all, TYPE);
    else p.sums[stretch * N + column] = all;
  }
}

// Rows to whole units; a checkpoint's to its values.
template <int TYPE>
__device__ __forceinline__ void prep_rows(const PrepRows& r, int64_t block, int64_t blocks) {
  const uint32_t per_row = (uint32_t)((r.K + 7) / 8);
  const int64_t all = r.R * per_row, scale_row = (r.K + 31) / 32;
  for (int64_t i = block * 256 + threadIdx.x; i < all; i += blocks * 256) {
    const int64_t row = over(i, per_row);
    const uint32_t c = (uint32_t)(i - row * per_row);
    const int64_t at = row * r.K + 8 * (int64_t)c, left = r.K - 8 * (int64_t)c;
    float v[8];
    if (r.scales) decode8(r.src, mx8_scale(r.scales[row * scale_row + (c >> 2)]), at, left < 8 ? (int)left : 8, v);
    else load8<TYPE>(r.src, at, left < 8 ? (int)left : 8, v);
    if (r.scales) hold8<TYPE>(v);
    store8<TYPE>(r.dst, 8 * i, 8, v);
  }
}

template <int TYPE>
__global__ __launch_bounds__(256) void prep_kernel(Prep p, int column_blocks, int act_blocks, int64_t rows, int L,
                                                   int blocks0, int blocks1) {
  __shared__ float meet[256 * 8];
#ifdef SWQ_LDS_POISON
  lds_poison(meet, sizeof(meet), kPoisonFloat);
  __syncthreads();
#endif
  int b = blockIdx.x;
  if (b < act_blocks) return act_backward<TYPE>(p, b % column_blocks, b / column_blocks, rows, L, meet);
  b -= act_blocks;
  if (b < blocks0) return prep_rows<TYPE>(p.rows[0], b, blocks0);
  prep_rows<TYPE>(p.rows[1], b - blocks0, blocks1);
}

__global__ __launch_bounds__(256) void zero16_kernel(uint16_t* p, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) p[i] = 0;
}

}  // namespace

hipError_t launch_mx8_quantize(const void* x, int64_t R, int64_t K, int type, void* codes, uint8_t* scales,
                               hipStream_t st) {
  return over_pieces(R, K, [&](dim3 grid, Pieces t, int64_t i, int64_t end) {
    if (type == kTypeF32) mx8_quantize_kernel<kTypeF32><<<grid, 256, 0, st>>>(x, t, i, end, codes, scales);
    else if (type == kTypeF16) mx8_quantize_kernel<kTypeF16><<<grid, 256, 0, st>>>(x, t, i, end, codes, scales);
    else mx8_quantize_kernel<kTypeBf16><<<grid, 256, 0, st>>>(x, t, i, end, codes, scales);
  });
}

hipError_t launch_mx8_dequantize(const void* codes, const uint8_t* scales, int64_t R, int64_t K, int type, void* out,
                                 hipStream_t st) {
  return over_pieces(R, K, [&](dim3 grid, Pieces t, int64_t i, int64_t end) {
    if (type == kTypeF32) mx8_dequantize_kernel<kTypeF32><<<grid, 256, 0, st>>>(codes, scales, t, i, end, out);
    else if (type == kTypeF16) mx8_dequantize_kernel<kTypeF16><<<grid, 256, 0, st>>>(codes, scales, t, i, end, out);
    else mx8_dequantize_kernel<kTypeBf16><<<grid, 256, 0, st>>>(codes, scales, t, i, end, out);
  });
}

hipError_t launch_swiglu(const uint16_t* gate, const uint16_t* up, int64_t R, int64_t K, int type, uint16_t* hidden,
                         void* gcodes, uint8_t* gscales, void* ucodes, uint8_t* uscales, hipStream_t st) {
  const auto kernel = type == kTypeF16 ? swiglu_kernel<kTypeF16> : swiglu_kernel<kTypeBf16>;
  return over_pieces(R, K, [&](dim3 grid, Pieces t, int64_t i, int64_t end) {
    kernel<<<grid, 256, 0, st>>>(gate, up, t, i, end, hidden, gcodes, gscales, ucodes, uscales);
  });
}

hipError_t launch_swiglu_backward(const uint16_t* dhidden, Kept gate, Kept up, int64_t R, int64_t K, int type,
                                  uint16_t* dgate, uint16_t* dup, uint16_t* hidden, hipStream_t st) {
  const auto kernel = type == kTypeF16 ? swiglu_backward_kernel<kTypeF16> : swiglu_backward_kernel<kTypeBf16>;
  return over_pieces(R, K, [&](dim3 grid, Pieces t, int64_t i, int64_t end) {
    kernel<<<grid, 256, 0, st>>>(dhidden, gate, up, t, i, end, dgate, dup, hidden);
  });
}

namespace {

// Lanes to a row, and stretches of rows: about 2048 blocks in all, four rows to a thread each at least; one up to
// sixteen rows.
int act_lanes(int64_t N) {
  int L = 1;
  while (L < 64 && 8 * L < N) L *= 2;
  return L;
}
int64_t act_rows(int64_t M, int64_t N) {
  const int L = act_lanes(N);
  const int64_t columns = (N + 8 * L - 1) / (8 * L), teams = 256 / L;
  if (M <= 16) return 16;
  const int64_t parts = std::max<int64_t>(1, std::min((M + 4 * teams - 1) / (4 * teams), 2048 / columns));
  return ((M + parts - 1) / parts + teams - 1) / teams * teams;
}

}  // namespace

int64_t act_parts(int64_t M, int64_t N) { return (M + act_rows(M, N) - 1) / act_rows(M, N); }

hipError_t launch_prep(const Prep& p, int type, hipStream_t st) {
  const int L = p.dout ? act_lanes(p.N) : 1;
  const int64_t columns = p.dout ? (p.N + 8 * L - 1) / (8 * L) : 0, parts = p.dout ? act_parts(p.M, p.N) : 0;
  const int64_t rows = p.dout ? act_rows(p.M, p.N) : 0;
  const auto blocks_for = [](const PrepRows& r) {
    return r.dst ? (int)std::min<int64_t>((r.R * ((r.K + 7) / 8) + 255) / 256, 4096) : 0;
  };
  const int n0 = blocks_for(p.rows[0]), n1 = blocks_for(p.rows[1]), act = (int)(columns * parts);
  if (act + n0 + n1 == 0) return hipSuccess;
  const auto kernel = type == kTypeF16 ? prep_kernel<kTypeF16> : prep_kernel<kTypeBf16>;
  kernel<<<(unsigned)(act + n0 + n1), 256, 0, st>>>(p, (int)columns, act, rows, L, n0, n1);
  return hipGetLastError();
}

hipError_t launch_zero16(uint16_t* p, int64_t n, hipStream_t st) {
  zero16_kernel<<<(unsigned)std::min<int64_t>((n + 255) / 256, 4096), 256, 0, st>>>(p, n);
  return hipGetLastError();
}

}  // namespace swq
