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

__device__ __forceinline__ void MxGemm::add_residual(float* f, int64_t at) const {
  if (!res) return;
  const u32x4 q = *(const u32x4*)(res + at);
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] += from_16((uint16_t)(q[i >> 1] >> (16 * (i & 1))), type);
}
__device__ __forceinline__ void MxGemm::add_one(float& f, int64_t at) const {
  if (res) f += from_16(res[at], type);
}

namespace {

constexpr int kTile = 16;
// A buffer offset past every buffer's end: the load returns zeros and touches no memory.
constexpr uint32_t kNowhere = 0xFFFFFFF0u;


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

// Sixteen rows of NT column tiles from a wave's accumulators (v[j]: lane 16 h + r has
// columns 16 j + 4 h .. + 3 of row r) to memory, through the wave's own stretch
// of LDS, so that a row leaves as whole lines: 16-byte stores of eight outputs (float32: two
// stores), or one output per lane where the rows are not aligned for that.
// row_at(i): the output row of the tile's row i; rows: how many there are.
constexpr int flush_floats(int nt) { return 16 * (16 * nt + 4); }
template <int NT, class Spec, class RowAt>
__device__ __forceinline__ void flush16(const Spec& p, float* buf, const f32x4* v, int rows, int col0, RowAt row_at) {
  constexpr int COLS = 16 * NT, LD = COLS + 4, UNITS = COLS / 8;
  const int lane = threadIdx.x & 63, r = lane & 15, h = lane >> 4;
  asm volatile("" ::: "memory");               // a wave's LDS accesses keep their order
#pragma unroll
  for (int j = 0; j < NT; ++j) *(f32x4*)(buf + r * LD + 16 * j + 4 * h) = v[j];
  asm volatile("" ::: "memory");
  if (p.vec == 2) {
#pragma unroll
    for (int i = 0; i < 16 * UNITS / 64; ++i) {
      const int u = i * 64 + lane, lr = u / UNITS, c = (u % UNITS) * 8, col = col0 + c;
      if (lr >= rows || col >= p.N) continue;
      const f32x4 a = *(const f32x4*)(buf + lr * LD + c), b = *(const f32x4*)(buf + lr * LD + c + 4);
      float f[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
      const int64_t at = row_at(lr) * p.N + col;
      p.add_residual(f, at);
      if (p.out_type == kTypeF32) {
        *(f32x4*)((float*)p.out + at) = (f32x4){f[0], f[1], f[2], f[3]};
        *(f32x4*)((float*)p.out + at + 4) = (f32x4){f[4], f[5], f[6], f[7]};
      } else {
        uint32_t q[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          q[e] = (uint32_t)to_16(f[2 * e], p.out_type) | (uint32_t)to_16(f[2 * e + 1], p.out_type) << 16;
        *(u32x4*)((uint16_t*)p.out + at) = (u32x4){q[0], q[1], q[2], q[3]};
        if (p.low_plane()) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            q[e] = (uint32_t)f32_to_bf16(bf16_rest(f[2 * e])) | (uint32_t)f32_to_bf16(bf16_rest(f[2 * e + 1])) << 16;
          *(u32x4*)(p.low_plane() + at) = (u32x4){q[0], q[1], q[2], q[3]};
        }
      }
    }
  } else {
#pragma unroll 1
    for (int u = lane; u < 16 * COLS; u += 64) {
      const int lr = u / COLS, c = u % COLS, col = col0 + c;
      if (lr >= rows || col >= p.N) continue;
      float f = buf[lr * LD + c];
      const int64_t at = row_at(lr) * p.N + col;
      p.add_one(f, at);
      if (p.out_type == kTypeF32) ((float*)p.out)[at] = f;
      else ((uint16_t*)p.out)[at] = to_16(f, p.out_type);
      if (p.low_plane()) p.low_plane()[at] = f32_to_bf16(bf16_rest(f));
    }
  }
}

// Four neighbouring sums of one output row: residual, rounding, store.
__device__ __forceinline__ void finish4(const MxGemm& p, int64_t at, int col, f32x4 v) {
  if (col >= p.N) return;
  if (p.hidden_planes) {
    f32x4 rest;
#pragma unroll
    for (int i = 0; i < 4; ++i) rest[i] = bf16_rest(v[i]);
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

// ----------------------------------------------------------- few-row kernel ----
//
// Up to 16 RT rows against 16 CT columns per block (SwiGLU: of both matrices).
// Here the weights' bytes count, not the sums: every wave takes chunks of
// 128 inputs c = wave, wave + W, ... on its own, weights and x straight to
// registers, U chunks of loads in flight, and the waves' sums meet in LDS at the
// end.  No barrier stands between the loads.
template <int RT, int CT, int XS, bool FUSED, int W, int U>
__device__ __forceinline__ void few_rows(const MxGemm& p, int expert, int first, int rows, int n0, f32x4* lds) {
  constexpr int NW = FUSED ? 2 * CT : CT, NP = XS == kXBf16 ? 1 : 2, NL = XS == kXPlanes ? 2 : 1;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, h = lane >> 4;
  f32x4 acc[RT][NW];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < NW; ++j) acc[i][j] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};

  if (expert >= 0) {
    // x: rows past the tile's read zeros and touch no memory
    const bool gather = p.xperm || p.ids;
    const uint16_t* xb = gather ? p.x : p.x + (int64_t)first * p.K;
    const uint32_t xbytes = (uint32_t)((int64_t)(gather ? p.xrows : rows) * p.K * 2);
    __amdgpu_buffer_rsrc_t xr[NL];
#pragma unroll
    for (int q = 0; q < NL; ++q)
      xr[q] = __builtin_amdgcn_make_buffer_rsrc((void*)(xb + q * p.plane), 0, (int)xbytes, 0x00020000);
    uint32_t xoff[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int lr = 16 * i + r;
      const int xrow = lr >= rows ? 0 : p.xperm ? p.xperm[first + lr] / p.xdiv : p.ids ? (first + lr) / p.xdiv : lr;
      xoff[i] = lr >= rows ? kNowhere : (uint32_t)xrow * (uint32_t)p.K * 2u + h * 64;
    }
    const int kb = p.K / 32, chunks = (kb + 3) / 4;
    const int64_t wrow = (int64_t)expert * p.N + n0;
    const int cols = p.N - n0;
    const int wbytes = min(cols, 16 * CT) * (p.K / 2);
    const __amdgpu_buffer_rsrc_t wr[2] = {
        __builtin_amdgcn_make_buffer_rsrc((void*)(p.w + wrow * (p.K / 8)), 0, wbytes, 0x00020000),
        __builtin_amdgcn_make_buffer_rsrc((void*)((FUSED ? p.w2 : p.w) + wrow * (p.K / 8)), 0, wbytes, 0x00020000)};
    const uint8_t* sb[2] = {p.s + wrow * kb, (FUSED ? p.s2 : p.s) + wrow * kb};

    for (int c0 = wave; c0 < chunks; c0 += W * U) {
      u32x4 w[U][NW], x[U][NL][RT][4];
      uint32_t s[U][NW];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = c0 + u * W;
        const bool in = 4 * c + h < kb;
#pragma unroll
        for (int j = 0; j < NW; ++j) {
          const int col = 16 * (j % CT) + r;
          w[u][j] = __builtin_bit_cast(
              u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                         wr[j / CT], in ? (uint32_t)col * (uint32_t)(p.K / 2) + c * 64 + h * 16 : kNowhere, 0, 0));
          s[u][j] = in ? sb[j / CT][(int64_t)min(col, cols - 1) * kb + 4 * c + h] : 0u;
        }
#pragma unroll
        for (int q = 0; q < NL; ++q)
#pragma unroll
          for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              x[u][q][i][k] = __builtin_bit_cast(
                  u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                             xr[q], in && xoff[i] != kNowhere ? xoff[i] + c * 256 + k * 16 : kNowhere, 0, 0));
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          bf16x8 a[NW];
#pragma unroll
          for (int j = 0; j < NW; ++j) a[j] = mx4_word(w[u][j][k], e8m0_operand(s[u][j]));
#pragma unroll
          for (int i = 0; i < RT; ++i) {
            bf16x8 b[NP];
            if constexpr (XS == kXF16) {
              split_f16x8(__builtin_bit_cast(f16x8, x[u][0][i][k]), b[0], b[NP - 1]);
            } else {
#pragma unroll
              for (int q = 0; q < NP; ++q) b[q] = __builtin_bit_cast(bf16x8, x[u][q % NL][i][k]);
            }
#pragma unroll
            for (int q = 0; q < NP; ++q)
#pragma unroll
              for (int j = 0; j < NW; ++j) acc[i][j] = mfma_bf16(a[j], b[q], acc[i][j]);
          }
        }
    }
  }

  // the waves' sums: [wave][i][j][lane], added in wave order
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < NW; ++j) lds[((wave * RT + i) * NW + j) * 64 + lane] = acc[i][j];
  __syncthreads();
  for (int f = wave; f < RT * CT; f += W) {
    const int i = f / CT, j = f % CT;
    f32x4 g = {0.0f, 0.0f, 0.0f, 0.0f}, u = g;
#pragma unroll
    for (int v = 0; v < W; ++v) {
      g += lds[((v * RT + i) * NW + j) * 64 + lane];
      if constexpr (FUSED) u += lds[((v * RT + i) * NW + j + CT) * 64 + lane];
    }
    if constexpr (FUSED) {
#pragma unroll
      for (int e = 0; e < 4; ++e) g[e] = silu_times(g[e], u[e]);
    }
    const int lr = 16 * i + r;
    if (lr < rows) {
      const int row = p.perm ? p.perm[first + lr] : first + lr;
      finish4(p, (int64_t)row * p.N, n0 + 16 * j + 4 * h, g);
    }
  }
}

// Rows of the block: a tile of the table, of a dense product, or the one row
// (slot) of p.ids.
template <int RT, int CT, int XS, bool FUSED, int W, int U>
__global__ __launch_bounds__(64 * W) void mx4_few_kernel(MxGemm p) {
  constexpr int F = RT * CT * (FUSED ? 2 : 1);
  __shared__ f32x4 lds[W * F * 64];
#ifdef SWQ_LDS_POISON
  lds_poison(lds, sizeof(lds), kPoisonFloat);
  __syncthreads();
#endif
  const int ntn = (p.N + 16 * CT - 1) / (16 * CT);
  int tm = blockIdx.x / ntn;
  const int tn = blockIdx.x - tm * ntn;
  int expert = 0, first = tm * 16 * RT, rows = min(16 * RT, p.rows - first);
  if (p.tiles) {
    if (tm >= *p.ntiles) return;
    const RowTile t = p.tiles[tm];
    expert = t.expert, first = t.first, rows = t.rows;
  } else if (p.ids) {
    expert = p.ids[tm], first = tm, rows = 1;
    if (expert < 0 || expert >= p.E) return;       // a skipped slot: nothing reads its row
  }
  expert = __builtin_amdgcn_readfirstlane(expert);
  first = __builtin_amdgcn_readfirstlane(first);
  rows = __builtin_amdgcn_readfirstlane(rows);
  if constexpr (RT > 1) {
    if (rows <= 16) return few_rows<1, CT, XS, FUSED, W, 2>(p, expert, first, rows, tn * 16 * CT, lds);
  }
  if constexpr (RT > 2) {
    if (rows <= 32) return few_rows<2, CT, XS, FUSED, W, 1>(p, expert, first, rows, tn * 16 * CT, lds);
  }
  few_rows<RT, CT, XS, FUSED, W, U>(p, expert, first, rows, tn * 16 * CT, lds);
}

// The experts' down projection of few tokens, one row each, with the weighted
// sum: block (token, 16 columns), wave v takes the token's slot v % k' and a share
// of its inputs, and the waves' sums, times the slots' weights, are added in
// wave order.  k' = k rounded up to a divisor or multiple of the W waves.
template <int XS, int W>
__global__ __launch_bounds__(64 * W) void mx4_down_kernel(MxGemm p, const float* __restrict__ weights, int k) {
  constexpr int NL = XS == kXPlanes ? 2 : 1;
  __shared__ f32x4 lds[W * 64];
#ifdef SWQ_LDS_POISON
  lds_poison(lds, sizeof(lds), kPoisonFloat);
  __syncthreads();
#endif
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, h = lane >> 4;
  const int ntn = (p.N + 15) / 16;
  const int t = blockIdx.x / ntn, n0 = (blockIdx.x - t * ntn) * 16;
  const int kb = p.K / 32, chunks = (kb + 3) / 4, cols = p.N - n0;
  // waves per slot: the largest power of two that leaves no slot waiting
  int share = W;
  while (share > 1 && share * k > W) share >>= 1;
  f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int j = wave / share; j < k; j += W / share) {
    const int slot = t * k + j;
    const int expert = __builtin_amdgcn_readfirstlane(p.ids[slot]);
    if (expert < 0 || expert >= p.E) continue;
    const float wt = weights[slot];
    const int64_t wrow = (int64_t)expert * p.N + n0;
    const __amdgpu_buffer_rsrc_t wr = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(p.w + wrow * (p.K / 8)), 0, min(cols, 16) * (p.K / 2), 0x00020000);
    const uint8_t* sb = p.s + (wrow + min(r, cols - 1)) * kb;
    __amdgpu_buffer_rsrc_t xr[NL];
#pragma unroll
    for (int q = 0; q < NL; ++q)
      xr[q] = __builtin_amdgcn_make_buffer_rsrc((void*)(p.x + q * p.plane + (int64_t)slot * p.K), 0, p.K * 2, 0x00020000);
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
    constexpr int U = 2;
    for (int c0 = wave % share; c0 < chunks; c0 += share * U) {
      u32x4 w[U], x[U][NL][4];
      uint32_t s[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = c0 + u * share;
        const bool in = 4 * c + h < kb;
        w[u] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                             wr, in ? (uint32_t)r * (uint32_t)(p.K / 2) + c * 64 + h * 16 : kNowhere, 0, 0));
        s[u] = in ? sb[4 * c + h] : 0u;
#pragma unroll
        for (int q = 0; q < NL; ++q)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            x[u][q][e] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                       xr[q], in && r == 0 ? c * 256 + h * 64 + e * 16 : kNowhere, 0, 0));
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const bf16x8 a = mx4_word(w[u][e], e8m0_operand(s[u]));
#pragma unroll
          for (int q = 0; q < NL; ++q) acc = mfma_bf16(a, __builtin_bit_cast(bf16x8, x[u][q][e]), acc);
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[e] = fmaf(wt, acc[e], sum[e]);
  }
  lds[wave * 64 + lane] = sum;
  __syncthreads();
  if (wave == 0 && r == 0) {
    f32x4 y = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int v = 0; v < W; ++v) y += lds[v * 64 + lane];
    finish4(p, (int64_t)t * p.N, n0 + 4 * h, y);
  }
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
#ifdef SWQ_LDS_POISON
  lds_poison(lds, sizeof(lds), kPoisonFloat);
  __syncthreads();
#endif
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
              in ? xoff[i] + (uint32_t)c * 256u : kNowhere);
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
            u32x4, __builtin_amdgcn_raw_buffer_load_b128(up ? wr1 : wr0, in ? woff[j] + c * 64 : kNowhere, 0, 0));
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

  // the stretches of the waves overlay the x buffers
  constexpr int NT = FUSED ? NF / 2 : NF;
  static_assert(flush_floats(NT) * W * 4 <= (int)sizeof(lds));
  float* buf = (float*)lds + wave * flush_floats(NT);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < MF; ++i) {
    const int r0 = (wm * MF + i) * 16;
    f32x4 v[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      v[j] = acc[i][j];
      if constexpr (FUSED) {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[j][e] = silu_times(v[j][e], acc[i][j + NF / 2][e]);
      }
    }
    flush16<NT>(p, buf, v, rows - r0, n0 + 16 * NT * wn, [&](int lr) {
      const int slot = first + r0 + lr;
      return (int64_t)(p.perm ? p.perm[slot] : slot);
    });
  }
}

// ----------------------------------------------------- two MXFP4 operands ----
//
// 16 x 16 x 128 scaled MFMA: lane 16 h + r holds row r's block h of a step of
// 128 inputs, 32 codes in four registers, and the byte of its scale operand
// that the step selects.
//
// The scales' bytes lie K / 32 apart, at any address, and a step needs four per row.  A first
// kernel lays them out as the MFMA takes them: for 16 rows and 512 inputs one
// word per lane, byte s for step s (blocks past K: 0).
__global__ __launch_bounds__(256) void mx4_scale_kernel(const uint8_t* __restrict__ sa, int M,
                                                        const uint8_t* __restrict__ sw, int N, int kb, int groups,
                                                        int pad_a, int pad_w, uint32_t* __restrict__ out) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;      // [row][group][h]
  const int h = (int)(i & 3);
  const int64_t rg = i >> 2;
  const int row = (int)(rg / groups), g = (int)(rg - (int64_t)row * groups);
  if (row >= pad_a + pad_w) return;
  const bool is_a = row < pad_a;
  const int at = is_a ? row : row - pad_a;
  const uint8_t* s = is_a ? sa : sw;
  uint32_t v = 0;
  if (at < (is_a ? M : N)) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int b = 16 * g + 4 * e + h;
      if (b < kb) v |= (uint32_t)s[(int64_t)at * kb + b] << (8 * e);
    }
  }
  out[((int64_t)(row / 16) * groups + g) * 64 + 16 * h + (row & 15)] = v;
}

// 256 x 256 outputs per block, 2 x 2 waves of 128 x 128.  A stage is one step,
// 256 rows of each operand (64 bytes a row), four stages in LDS; a step reads its
// successor's operands into registers while its MFMAs run and starts the
// loads of the stage four ahead.  16-byte unit h of a row sits at
// h ^ (row / 4 & 3): the sixteen rows of a read lie in different banks.
constexpr int kMmTile = 256, kMmStage = 2 * kMmTile * 64, kMmScales = 2 * kMmTile * 16;

__global__ __launch_bounds__(256, 1) void mx4_matmul_kernel(Mx4Matmul p, const uint32_t* __restrict__ scales,
                                                            int groups, int pad_a) {
  __shared__ __attribute__((aligned(1024))) char lds[4 * kMmStage + 2 * kMmScales];
#ifdef SWQ_LDS_POISON
  lds_poison(lds, sizeof(lds), kPoisonFloat);
  __syncthreads();
#endif
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, h = lane >> 4;
  const int wm = wave >> 1, wn = wave & 1;
  int tm, tn;
  if (!tile_of(blockIdx.x, (p.M + kMmTile - 1) / kMmTile, (p.N + kMmTile - 1) / kMmTile, tm, tn)) return;
  const int m0 = tm * kMmTile, n0 = tn * kMmTile;
  const int steps = (p.K + 127) / 128, row_bytes = p.K / 2;

  // codes: wave w loads rows 16 (4 i + w) + lane / 4 of each operand, a row past the
  // end repeating the tile's first
  const int rows_a = min(kMmTile, p.M - m0), rows_w = min(kMmTile, p.N - n0);
  const i32x4 ra = make_srsrc((const char*)p.a + (int64_t)m0 * row_bytes, (uint32_t)rows_a * row_bytes);
  const i32x4 rw = make_srsrc((const char*)p.w + (int64_t)n0 * row_bytes, (uint32_t)rows_w * row_bytes);
  const int lrow = wave * 16 + (lane >> 2);
  const int unit = (lane & 3) ^ (lane >> 4);           // (row / 4 & 3) == lane / 16
  uint32_t offa[4], offw[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = 64 * i + lrow;
    offa[i] = (uint32_t)(row < rows_a ? row : 0) * row_bytes + unit * 16;
    offw[i] = (uint32_t)(row < rows_w ? row : 0) * row_bytes + unit * 16;
  }
  const uint32_t lds0 = lds_addr(lds);
  const auto stage = [&](int t, int slot) {
    const bool in = t * 128 + unit * 32 < p.K;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t base = __builtin_amdgcn_readfirstlane(lds0 + slot * kMmStage + (i * 4 + wave) * 1024);
      dma16(ra, base, in ? offa[i] + (uint32_t)t * 64u : kNowhere);
      dma16(rw, base + kMmTile * 64, in ? offw[i] + (uint32_t)t * 64u : kNowhere);
    }
  };
  // scales of a group of four steps: 16 row groups of 256 bytes for each operand, gathered
  // 1 KB per load: lane l takes 16 bytes of row group 4 w + l / 16
  const i32x4 rsa = make_srsrc(scales + (int64_t)(m0 / 16) * groups * 64, (uint32_t)(16 * groups * 256));
  const i32x4 rsw = make_srsrc(scales + (int64_t)((pad_a + n0) / 16) * groups * 64, (uint32_t)(16 * groups * 256));
  const uint32_t soff = (uint32_t)(4 * wave + (lane >> 4)) * groups * 256 + (lane & 15) * 16;
  const auto stage_scales = [&](int g) {
    const uint32_t base = __builtin_amdgcn_readfirstlane(lds0 + 4 * kMmStage + (g & 1) * kMmScales + wave * 1024);
    dma16(rsa, base, g < groups ? soff + g * 256 : kNowhere);
    dma16(rsw, base + kMmTile * 16, g < groups ? soff + g * 256 : kNowhere);
  };

  f32x4 acc[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};

  const uint32_t frag = r * 64 + ((h ^ (r >> 2)) * 16);
  u32x4 a[2][8], w[2][8];
  uint32_t sa[8], sw[8];
  const auto read_codes = [&](int slot, u32x4* fa, u32x4* fw) {
    const char* s = lds + slot * kMmStage + frag;
#pragma unroll
    for (int i = 0; i < 8; ++i) fa[i] = *(const u32x4*)(s + (wm * 8 + i) * 1024);
#pragma unroll
    for (int j = 0; j < 8; ++j) fw[j] = *(const u32x4*)(s + kMmTile * 64 + (wn * 8 + j) * 1024);
  };
  const auto read_scales = [&](int g, uint32_t* fa, uint32_t* fw) {
    const char* s = lds + 4 * kMmStage + (g & 1) * kMmScales + lane * 4;
#pragma unroll
    for (int i = 0; i < 8; ++i) fa[i] = *(const uint32_t*)(s + (wm * 8 + i) * 256);
#pragma unroll
    for (int j = 0; j < 8; ++j) fw[j] = *(const uint32_t*)(s + kMmTile * 16 + (wn * 8 + j) * 256);
  };
  const auto meet = [&]() {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };

  stage_scales(0);
#pragma unroll
  for (int t = 0; t < 4; ++t) stage(t, t);
  wait_vmcnt<24>();
  meet();
  read_codes(0, a[0], w[0]);

  // One step.  Loads are issued past the last step too (they read nothing), so the counts below hold to the end.
  const auto step = [&]<int CUR>(int t) {
    constexpr int NXT = CUR ^ 1;
    wait_vmcnt<16>();          // all but the last two stages' loads: stage t + 1 is there
    meet();
    if ((t & 3) == 0) {
      read_scales(t >> 2, sa, sw);
      stage_scales((t >> 2) + 1);
    }
    stage(t + 4, t & 3);
    read_codes((t + 1) & 3, a[NXT], w[NXT]);
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[i][j] = mfma_mx4(w[CUR][j], sw[j], a[CUR][i], sa[i], acc[i][j]);
#pragma unroll
    for (int i = 0; i < 8; ++i) sa[i] >>= 8, sw[i] >>= 8;
  };
  for (int t = 0; t < steps; t += 2) {
    step.template operator()<0>(t);
    step.template operator()<1>(t + 1);
  }
  wait_vmcnt<0>();             // no load may write LDS after the block has left

  meet();                      // the waves' stretches overlay the stages
  float* buf = (float*)lds + wave * flush_floats(8);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r0 = m0 + (wm * 8 + i) * 16;
    flush16<8>(p, buf, acc[i], p.M - r0, n0 + wn * 128, [&](int lr) { return (int64_t)(r0 + lr); });
  }
}

// Few rows: one wave per 16 x 16 outputs, everything straight to registers.
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
  if (n0 + 4 * h < p.N) store4(p.out, m * p.N, n0 + 4 * h, p.N, p.vec, acc, p.out_type);
}

}  // namespace

// Kernel of a product: the few-row kernel below a row count, else the tiled one.
// A grouped product goes by its rows per expert.
static bool few(const MxGemm& p) {
  if (const char* e = getenv("SWQ_MX4_FEW")) return p.rows / p.E < atoi(e);
  return p.rows / p.E < 64;
}

static int few_tiles(const MxGemm& p) {       // row tiles of 16 of the few-row kernel
  if (p.ids && !p.tiles) return 1;
  return p.tiles ? 4 : p.rows <= 16 ? 1 : p.rows <= 32 ? 2 : 4;
}

int mx4_gemm_tile(const MxGemm& p) {
  if (few(p)) return 64;
  return p.xsrc != kXBf16 ? 64 : 128;
}

bool mx4_gemm_takes_planes(const MxGemm& p) { return !few(p); }

template <int MF, int NF, int WM, int WN, int NP, bool FUSED>
static hipError_t launch_tiled(const MxGemm& p, hipStream_t st) {
  constexpr int BM = 16 * MF * WM, BNO = 16 * NF * WN / (FUSED ? 2 : 1);
  const int64_t ntm = p.tiles ? p.max_tiles : (p.rows + BM - 1) / BM, ntn = (p.N + BNO - 1) / BNO;
  const int64_t blocks = (ntm * ntn + 7) / 8 * 8;
  if (blocks >= (1LL << 31)) return hipErrorInvalidValue;
  mx4_gemm_kernel<MF, NF, WM, WN, NP, FUSED><<<dim3((unsigned)blocks), 64 * WM * WN, 0, st>>>(p);
  return hipGetLastError();
}

template <int RT, int CT, int XS, bool FUSED, int W, int U>
static hipError_t launch_few_as(const MxGemm& p, hipStream_t st) {
  const int64_t ntn = (p.N + 16 * CT - 1) / (16 * CT);
  const int64_t ntm = p.tiles ? p.max_tiles : p.ids ? p.rows : (p.rows + 16 * RT - 1) / (16 * RT);
  if (ntm * ntn >= (1LL << 31)) return hipErrorInvalidValue;
  mx4_few_kernel<RT, CT, XS, FUSED, W, U><<<dim3((unsigned)(ntm * ntn)), 64 * W, 0, st>>>(p);
  return hipGetLastError();
}

template <int XS, bool FUSED>
static hipError_t launch_few(const MxGemm& p, hipStream_t st) {
  const int rt = few_tiles(p);
  if (rt == 1) return launch_few_as<1, 1, XS, FUSED, 8, 2>(p, st);
  if (rt == 2) return launch_few_as<2, FUSED ? 1 : 2, XS, FUSED, 8, 1>(p, st);
  return launch_few_as<4, FUSED ? 1 : 2, XS, FUSED, 8, 1>(p, st);
}

hipError_t launch_mx4_gemm(const MxGemm& p, hipStream_t st) {
  const bool fused = p.w2;
  if ((p.ids && !p.tiles) || few(p)) {
    if (p.xsrc == kXBf16) return fused ? launch_few<kXBf16, true>(p, st) : launch_few<kXBf16, false>(p, st);
    if (p.xsrc == kXF16) return fused ? launch_few<kXF16, true>(p, st) : launch_few<kXF16, false>(p, st);
    return fused ? launch_few<kXPlanes, true>(p, st) : launch_few<kXPlanes, false>(p, st);
  }
  if (p.xsrc != kXBf16) return fused ? launch_tiled<4, 4, 1, 4, 2, true>(p, st) : launch_tiled<4, 4, 1, 4, 2, false>(p, st);
  return fused ? launch_tiled<8, 4, 1, 4, 1, true>(p, st) : launch_tiled<8, 4, 1, 4, 1, false>(p, st);
}

hipError_t launch_mx4_down(const MxGemm& p, const float* weights, int k, hipStream_t st) {
  const int64_t blocks = (int64_t)(p.rows / k) * ((p.N + 15) / 16);
  if (blocks >= (1LL << 31)) return hipErrorInvalidValue;
  if (p.xsrc == kXPlanes) mx4_down_kernel<kXPlanes, 16><<<dim3((unsigned)blocks), 1024, 0, st>>>(p, weights, k);
  else mx4_down_kernel<kXBf16, 16><<<dim3((unsigned)blocks), 1024, 0, st>>>(p, weights, k);
  return hipGetLastError();
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

static int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

int64_t mx4_matmul_workspace(const Mx4Matmul& p) {
  if (p.M < 64) return 0;
  return (round_up(p.M, kMmTile) + round_up(p.N, kMmTile)) * ((p.K + 511) / 512) * 16;
}

hipError_t launch_mx4_matmul(const Mx4Matmul& p, void* ws, hipStream_t st) {
  if (!ws) {
    const int64_t tiles = (int64_t)((p.N + kTile - 1) / kTile) * ((p.M + kTile - 1) / kTile);
    if (tiles >= (1LL << 31)) return hipErrorInvalidValue;
    mx4_matmul_tile_kernel<<<dim3((unsigned)tiles), 64, 0, st>>>(p);
    return hipGetLastError();
  }
  const int groups = (p.K + 511) / 512;
  const int pad_a = (int)round_up(p.M, kMmTile), pad_w = (int)round_up(p.N, kMmTile);
  const int64_t words = (int64_t)(pad_a + pad_w) * groups * 4;
  mx4_scale_kernel<<<dim3((unsigned)((words + 255) / 256)), 256, 0, st>>>(p.sa, p.M, p.s, p.N, p.K / 32, groups, pad_a,
                                                                        pad_w, (uint32_t*)ws);
  const int64_t tiles = (int64_t)(pad_a / kMmTile) * (pad_w / kMmTile);
  if (tiles >= (1LL << 30)) return hipErrorInvalidValue;
  mx4_matmul_kernel<<<dim3((unsigned)round_up(tiles, 8)), 256, 0, st>>>(p, (const uint32_t*)ws, groups, pad_a);
  return hipGetLastError();
}

}  // namespace swq
