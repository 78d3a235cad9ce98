// Products with MXFP4 weights: y = x W^T for bf16 or binary16 x, dense or grouped
// by expert, plain or as the SwiGLU of two such products, and the product of
// two MXFP4 operands.
//
// A bf16 MFMA of 16 x 16 x 32 takes eight inputs per lane: lane 16 h + r holds
// row r's inputs [8 h, 8 h + 8) of a K-step of 32, which is one word of codes and
// one scale block, so a weight operand is one converted word.  The weights are
// the first operand: lane 16 h + r of the result holds columns 4 h .. 4 h + 3 of
// row r, four neighbours for one store.  The products are exact (8 by 2
// significant bits); only the float32 sums and the last rounding are not.
// binary16 rows are split into two bf16 operands (split_f16), exact too.
#include "swq_mx4.h"
#include "swq_mx4_device.h"

namespace swq {
namespace {

constexpr int kTile = 16;

__device__ __forceinline__ void load_x(const MxGemm& p, int64_t at, bf16x8& hi, bf16x8& lo) {
  if (p.xsrc == kXF16) {
    split_f16x8(*(const f16x8*)(p.x + at), hi, lo);
  } else {
    hi = *(const bf16x8*)(p.x + at);
    if (p.xsrc == kXPlanes) lo = *(const bf16x8*)(p.x + p.plane + at);
  }
}

// One wave per 16 x 16 outputs.
__global__ __launch_bounds__(64) void mx4_tile_kernel(MxGemm p) {
  const int lane = threadIdx.x, r = lane & 15, h = lane >> 4;
  const int ntn = (p.N + kTile - 1) / kTile;
  const int tm = blockIdx.x / ntn, n0 = (blockIdx.x % ntn) * kTile;
  int expert = 0, first = tm * kTile, rows = min(kTile, p.rows - first);
  if (p.tiles) {
    if (tm >= *p.ntiles) return;
    const RowTile t = p.tiles[tm];
    expert = t.expert, first = t.first, rows = t.rows;
  }
  const int n = min(n0 + r, p.N - 1);
  const int slot = first + min(r, rows - 1);
  const int row = p.perm ? p.perm[slot] : slot;
  const int64_t xat = (int64_t)(row / p.xdiv) * p.K;
  f32x4 g = {}, u = {};
  if (expert >= 0) {
    const int64_t wrow = (int64_t)expert * p.N + n;
    const bool two = p.xsrc != kXBf16;
    for (int kb = 0; kb < p.K / 32; ++kb) {
      bf16x8 hi, lo;
      load_x(p, xat + kb * 32 + 8 * h, hi, lo);
      const int64_t word = wrow * (p.K / 8) + kb * 4 + h, sc = wrow * (p.K / 32) + kb;
      const bf16x8 a = mx4_word(p.w[word], e8m0_operand(p.s[sc]));
      g = mfma_bf16(a, hi, g);
      if (two) g = mfma_bf16(a, lo, g);
      if (p.w2) {
        const bf16x8 b = mx4_word(p.w2[word], e8m0_operand(p.s2[sc]));
        u = mfma_bf16(b, hi, u);
        if (two) u = mfma_bf16(b, lo, u);
      }
    }
  }
  if (r >= rows) return;
  const int col = n0 + 4 * h;
  if (p.w2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) g[i] = silu_times(g[i], u[i]);
  }
  const int64_t at = (int64_t)row * p.N;
  if (p.hidden_planes) {
    f32x4 rest;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float hi = round_to_bf16(g[i]);
      rest[i] = __builtin_isfinite(hi) ? g[i] - hi : 0.0f;
    }
    store4(p.out, at, col, p.N, false, g, kTypeBf16);
    store4((uint16_t*)p.out + p.out_plane, at, col, p.N, false, rest, kTypeBf16);
    return;
  }
  if (p.res) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (col + i < p.N) g[i] += from_16(p.res[at + col + i], p.type);
  }
  store4(p.out, at, col, p.N, false, g, p.out_type);
}

// Both operands MXFP4: 16 x 16 x 128 scaled MFMA, one block of 32 per lane.
__global__ __launch_bounds__(64) void mx4_matmul_tile_kernel(Mx4Matmul p) {
  const int lane = threadIdx.x, r = lane & 15, h = lane >> 4;
  const int ntn = (p.N + kTile - 1) / kTile;
  const int m0 = (blockIdx.x / ntn) * kTile, n0 = (blockIdx.x % ntn) * kTile;
  const int64_t n = min(n0 + r, p.N - 1), m = min(m0 + r, p.M - 1);
  const int blocks = p.K / 32;
  f32x4 acc = {};
  for (int kb = 0; kb < blocks; kb += 4) {
    u32x4 a = {}, w = {};
    uint32_t sa = 0, sw = 0;
    if (kb + h < blocks) {
      a = ((const u32x4*)p.a)[m * blocks + kb + h];
      w = ((const u32x4*)p.w)[n * blocks + kb + h];
      sa = p.sa[m * blocks + kb + h];
      sw = p.s[n * blocks + kb + h];
    }
    acc = mfma_mx4(w, sw, a, sa, acc);
  }
  if (m0 + r >= p.M) return;
  store4(p.out, m * p.N, n0 + 4 * h, p.N, false, acc, p.out_type);
}

}  // namespace

int mx4_gemm_tile(const MxGemm&) { return kTile; }

hipError_t launch_mx4_gemm(const MxGemm& p, hipStream_t st) {
  const int64_t ntn = (p.N + kTile - 1) / kTile;
  const int64_t ntm = p.tiles ? p.max_tiles : (p.rows + kTile - 1) / kTile;
  if (ntn * ntm >= (1LL << 31)) return hipErrorInvalidValue;
  mx4_tile_kernel<<<dim3((unsigned)(ntn * ntm)), 64, 0, st>>>(p);
  return hipGetLastError();
}

hipError_t launch_mx4_matmul(const Mx4Matmul& p, hipStream_t st) {
  const int64_t tiles = (int64_t)((p.N + kTile - 1) / kTile) * ((p.M + kTile - 1) / kTile);
  if (tiles >= (1LL << 31)) return hipErrorInvalidValue;
  mx4_matmul_tile_kernel<<<dim3((unsigned)tiles), 64, 0, st>>>(p);
  return hipGetLastError();
}

}  // namespace swq
