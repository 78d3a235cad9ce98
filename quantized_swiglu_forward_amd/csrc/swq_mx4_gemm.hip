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
#include <stdlib.h>

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


// XCD-aware order of the tiles: the hardware deals consecutive blocks to the
// eight XCDs in turn, so block b takes tile b / 8 of a contiguous eighth of the
// order, and an XCD's own L2 sees neighbours.  In the order, bands of eight row
// tiles run down their columns.  False: nothing for this block.
__device__ __forceinline__ bool tile_of(int b, int ntm, int ntn, int& tm, int& tn) {
  const int total = ntm * ntn, per = (total + 7) / 8;
  const int t = (b & 7) * per + (b >> 3);
  if ((b >> 3) >= per || t >= total) return false;
  const int band = t / (8 * ntn), in = t - band * 8 * ntn, high = min(8, ntm - 8 * band);
  tm = 8 * band + in % high;
  tn = in / high;
  return true;
}

// Four neighbouring sums of one output row: residual, rounding, store.
__device__ __forceinline__ void finish4(const MxGemm& p, int64_t at, int col, f32x4 v) {
  if (col >= p.N) return;
  if (p.hidden_planes) {
    f32x4 rest;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float hi = round_to_bf16(v[i]);
      rest[i] = __builtin_isfinite(hi) ? v[i] - hi : 0.0f;
    }
    store4(p.out, at, col, p.N, p.vec, v, kTypeBf16);
    store4((uint16_t*)p.out + p.out_plane, at, col, p.N, p.vec, rest, kTypeBf16);
    return;
  }
  if (p.res) {
    if (p.vec && col + 4 <= p.N) {
      const u32x2 q = *(const u32x2*)(p.res + at + col);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += from_16((uint16_t)(q[i >> 1] >> (16 * (i & 1))), p.type);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (col + i < p.N) v[i] += from_16(p.res[at + col + i], p.type);
    }
  }
  store4(p.out, at, col, p.N, p.vec, v, p.out_type);
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
  const int64_t xat = (int64_t)(p.xperm ? p.xperm[slot] / p.xdiv : slot) * p.K;
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
  if (p.w2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) g[i] = silu_times(g[i], u[i]);
  }
  finish4(p, (int64_t)(p.perm ? p.perm[slot] : slot) * p.N, n0 + 4 * h, g);
}

// ------------------------------------------------------------ tiled kernel ----
//
// WM x WN waves, each MF x NF accumulators of 16 x 16 over 16 MF rows of x and
// 16 NF columns of W (SwiGLU: NF / 2 column tiles of the gate and the same of the
// up matrix).  A chunk is 128 inputs: lane 16 h + r takes block h of a chunk
// in four steps, so its codes are one 16-byte load and its scale one byte,
// straight from memory to registers one chunk ahead (a column's codes are used
// by WM waves only).  x goes through LDS, [BM * NP][128] bf16, two buffers, by
// loads that write LDS; 16-byte unit u of a row sits at u ^ (row & 15), so the
// sixteen rows that a read touches lie in different banks.
template <int MF, int NF, int WM, int WN, int NP, bool FUSED>
__global__ __launch_bounds__(64 * WM * WN, 2) void mx4_gemm_kernel(MxGemm p) {
  constexpr int W = WM * WN, BM = 16 * MF * WM, ROWS = BM * NP, BN = 16 * NF * WN, BNO = FUSED ? BN / 2 : BN;
  constexpr int DMA = ROWS / (4 * W);           // loads per lane and chunk, four rows each per wave
  static_assert(ROWS % (4 * W) == 0 && (!FUSED || NF % 2 == 0));
  __shared__ __attribute__((aligned(1024))) char lds[2][ROWS * 256];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, h = lane >> 4;
  const int wm = wave / WN, wn = wave % WN;

  const int ntn = (p.N + BNO - 1) / BNO;
  int tm, tn;
  if (!tile_of(blockIdx.x, p.tiles ? *p.ntiles : (p.rows + BM - 1) / BM, ntn, tm, tn)) return;
  int expert = 0, first = tm * BM, rows = min(BM, p.rows - first);
  if (p.tiles) {
    const RowTile t = p.tiles[tm];
    expert = __builtin_amdgcn_readfirstlane(t.expert);
    first = __builtin_amdgcn_readfirstlane(t.first);
    rows = __builtin_amdgcn_readfirstlane(t.rows);
  }
  const int n0 = tn * BNO;

  f32x4 acc[MF][NF];
#pragma unroll
  for (int i = 0; i < MF; ++i)
#pragma unroll
    for (int j = 0; j < NF; ++j) acc[i][j] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};

  const int chunks = (p.K + 127) / 128;
  if (expert >= 0) {
    // x: rows of the tile from its first (contiguous rows) or from row 0 (gathered)
    const uint16_t* xb = p.xperm ? p.x : p.x + (int64_t)first * p.K;
    const int64_t xbytes = p.xperm ? (int64_t)p.xrows * p.K * 2 : (int64_t)rows * p.K * 2;
    i32x4 xr[NP];
#pragma unroll
    for (int q = 0; q < NP; ++q) xr[q] = make_srsrc(xb + q * p.plane, (uint32_t)xbytes);
    const int drow = wave * 4 + (lane >> 4);
    const int du = (lane & 15) ^ (drow & 15);   // the unit that this lane loads, in each of its rows
    uint32_t xoff[DMA];
#pragma unroll
    for (int i = 0; i < DMA; ++i) {
      const int lr = (i * 4 * W + drow) % BM;
      const int slot = lr < rows ? lr : 0;      // rows past the tile's repeat its first
      const int xrow = p.xperm ? p.xperm[first + slot] / p.xdiv : slot;
      xoff[i] = (uint32_t)xrow * (uint32_t)p.K * 2u + du * 16;
    }
    const auto stage = [&](int c, int buf) {
      const bool in = c * 128 + du * 8 < p.K;   // past K: zeros
#pragma unroll
      for (int i = 0; i < DMA; ++i) {
        const uint32_t base = lds_addr(&lds[buf][(i * 4 * W + wave * 4) * 256]);
        dma16(xr[(i * 4 * W) / BM], __builtin_amdgcn_readfirstlane(base),
              in ? xoff[i] + (uint32_t)c * 256u : 0xFFFFFFF0u);
      }
    };

    // W: the columns of this wave; rows past N read zeros
    const int kb = p.K / 32;
    const int64_t wrow = (int64_t)expert * p.N + n0;
    const int wn_rows = p.N - n0;
    uint32_t woff[NF];
    int scol[NF];
#pragma unroll
    for (int j = 0; j < NF; ++j) {
      const int col = FUSED ? 16 * (wn * (NF / 2) + j % (NF / 2)) + r : 16 * (wn * NF + j) + r;
      woff[j] = (uint32_t)col * (uint32_t)(p.K / 2) + h * 16;
      scol[j] = min(col, wn_rows - 1);
    }
    const __amdgpu_buffer_rsrc_t wr0 = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(p.w + wrow * (p.K / 8)), 0, (int)min((int64_t)wn_rows, (int64_t)BNO) * (p.K / 2), 0x00020000);
    const __amdgpu_buffer_rsrc_t wr1 = __builtin_amdgcn_make_buffer_rsrc(
        (void*)((FUSED ? p.w2 : p.w) + wrow * (p.K / 8)), 0, (int)min((int64_t)wn_rows, (int64_t)BNO) * (p.K / 2),
        0x00020000);
    const uint8_t* s0 = p.s + wrow * kb;
    const uint8_t* s1 = (FUSED ? p.s2 : p.s) + wrow * kb;
    u32x4 wc[NF];
    uint32_t sc[NF];
    const auto load_w = [&](int c, u32x4* w, uint32_t* s) {
      const bool in = 4 * c + h < kb;
#pragma unroll
      for (int j = 0; j < NF; ++j) {
        const bool up = FUSED && j >= NF / 2;
        w[j] = __builtin_bit_cast(
            u32x4, __builtin_amdgcn_raw_buffer_load_b128(up ? wr1 : wr0, in ? woff[j] + c * 64 : 0xFFFFFFF0u, 0, 0));
        s[j] = in ? (up ? s1 : s0)[(int64_t)scol[j] * kb + 4 * c + h] : 0u;
      }
    };

    stage(0, 0);
    load_w(0, wc, sc);
    wait_vmcnt<0>();
    __syncthreads();
    int buf = 0;
    for (int c = 0; c < chunks; ++c) {
      u32x4 wnext[NF];
      uint32_t snext[NF];
      const bool more = c + 1 < chunks;
      if (more) {
        stage(c + 1, buf ^ 1);
        load_w(c + 1, wnext, snext);
      }
      const char* xt = lds[buf] + (wm * MF * 16 + r) * 256;
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        bf16x8 a[NF];
#pragma unroll
        for (int j = 0; j < NF; ++j) a[j] = mx4_word(wc[j][s], e8m0_operand(sc[j]));
        const char* xu = xt + (((4 * h + s) ^ r) * 16);
#pragma unroll
        for (int q = 0; q < NP; ++q)
#pragma unroll
          for (int i = 0; i < MF; ++i) {
            const bf16x8 b = *(const bf16x8*)(xu + (q * BM + 16 * i) * 256);
#pragma unroll
            for (int j = 0; j < NF; ++j) acc[i][j] = mfma_bf16(a[j], b, acc[i][j]);
          }
      }
      if (more) {
#pragma unroll
        for (int j = 0; j < NF; ++j) wc[j] = wnext[j], sc[j] = snext[j];
        wait_vmcnt<0>();
        __syncthreads();
        buf ^= 1;
      }
    }
  }

#pragma unroll
  for (int i = 0; i < MF; ++i) {
    const int lr = (wm * MF + i) * 16 + r;
    if (lr >= rows) continue;
    const int row = p.perm ? p.perm[first + lr] : first + lr;
    const int64_t at = (int64_t)row * p.N;
#pragma unroll
    for (int j = 0; j < (FUSED ? NF / 2 : NF); ++j) {
      const int col = n0 + 16 * (FUSED ? wn * (NF / 2) + j : wn * NF + j) + 4 * h;
      f32x4 v = acc[i][j];
      if constexpr (FUSED) {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = silu_times(v[e], acc[i][j + NF / 2][e]);
      }
      finish4(p, at, col, v);
    }
  }
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

// Tile shapes (rows): 0 the simple kernel, else the tiled one.
struct GemmConfig {
  int bm, bno;
};
}  // namespace

static int pick(const MxGemm& p) {
  if (const char* e = getenv("SWQ_MX4_CFG")) return atoi(e);
  return p.rows <= 16 ? 0 : 1;
}
static bool planes_of(const MxGemm& p) { return p.xsrc != kXBf16; }

int mx4_gemm_tile(const MxGemm& p) {
  const int c = pick(p);
  if (c == 0) return 16;
  const int bm = c == 3 ? 256 : c == 2 ? 128 : 64;
  return planes_of(p) && bm == 256 ? 128 : bm;
}

bool mx4_gemm_takes_planes(const MxGemm& p) { return pick(p) != 0; }

template <int MF, int NF, int WM, int WN, int NP, bool FUSED>
static hipError_t launch_tiled(const MxGemm& p, hipStream_t st) {
  constexpr int BM = 16 * MF * WM, BNO = 16 * NF * WN / (FUSED ? 2 : 1);
  const int64_t ntm = p.tiles ? p.max_tiles : (p.rows + BM - 1) / BM, ntn = (p.N + BNO - 1) / BNO;
  const int64_t blocks = (ntm * ntn + 7) / 8 * 8;
  if (blocks >= (1LL << 31)) return hipErrorInvalidValue;
  mx4_gemm_kernel<MF, NF, WM, WN, NP, FUSED><<<dim3((unsigned)blocks), 64 * WM * WN, 0, st>>>(p);
  return hipGetLastError();
}

hipError_t launch_mx4_gemm(const MxGemm& p, hipStream_t st) {
  const int c = pick(p);
  if (c == 0) {
    const int64_t ntn = (p.N + kTile - 1) / kTile;
    const int64_t ntm = p.tiles ? p.max_tiles : (p.rows + kTile - 1) / kTile;
    if (ntn * ntm >= (1LL << 31)) return hipErrorInvalidValue;
    mx4_tile_kernel<<<dim3((unsigned)(ntn * ntm)), 64, 0, st>>>(p);
    return hipGetLastError();
  }
  const bool two = planes_of(p), fused = p.w2;
  if (c == 1) {
    if (two) return fused ? launch_tiled<4, 2, 1, 8, 2, true>(p, st) : launch_tiled<4, 2, 1, 8, 2, false>(p, st);
    return fused ? launch_tiled<4, 2, 1, 8, 1, true>(p, st) : launch_tiled<4, 2, 1, 8, 1, false>(p, st);
  }
  if (two) return fused ? launch_tiled<4, 4, 2, 4, 2, true>(p, st) : launch_tiled<4, 4, 2, 4, 2, false>(p, st);
  if (c == 2) return fused ? launch_tiled<4, 4, 2, 4, 1, true>(p, st) : launch_tiled<4, 4, 2, 4, 1, false>(p, st);
  return fused ? launch_tiled<8, 4, 2, 4, 1, true>(p, st) : launch_tiled<8, 4, 2, 4, 1, false>(p, st);
}

namespace {
__global__ __launch_bounds__(256) void mx4_split_kernel(const f16x8* __restrict__ x, int64_t n8,
                                                        bf16x8* __restrict__ hi, bf16x8* __restrict__ lo) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n8) return;
  bf16x8 a, b;
  split_f16x8(x[i], a, b);
  hi[i] = a;
  lo[i] = b;
}
}  // namespace

hipError_t launch_mx4_split(const uint16_t* x, int64_t n, uint16_t* planes, int64_t plane, hipStream_t st) {
  mx4_split_kernel<<<dim3((unsigned)((n / 8 + 255) / 256)), 256, 0, st>>>((const f16x8*)x, n / 8, (bf16x8*)planes,
                                                                         (bf16x8*)(planes + plane));
  return hipGetLastError();
}

hipError_t launch_mx4_matmul(const Mx4Matmul& p, hipStream_t st) {
  const int64_t tiles = (int64_t)((p.N + kTile - 1) / kTile) * ((p.M + kTile - 1) / kTile);
  if (tiles >= (1LL << 31)) return hipErrorInvalidValue;
  mx4_matmul_tile_kernel<<<dim3((unsigned)tiles), 64, 0, st>>>(p);
  return hipGetLastError();
}

}  // namespace swq
