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
#include <algorithm>

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

// A buffer offset past every buffer's end: the load returns zeros and touches no memory.
constexpr uint32_t kNowhere = 0xFFFFFFF0u;

// Loads through a buffer descriptor.  What is out of range is asked for at
// kNowhere instead of being branched around: a branch around a load makes the
// compiler wait for every load in flight where the paths meet.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc((void*)base, 0, (int)bytes, 0x00020000);
}
__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t b, uint32_t off) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(b, off, 0, 0));
}
__device__ __forceinline__ uint32_t load1(__amdgpu_buffer_rsrc_t b, uint32_t off) {
  return __builtin_amdgcn_raw_buffer_load_b8(b, off, 0, 0);
}


// f.operator()<0>(), f.operator()<1>(), ...
template <int N, int I = 0, class F>
__device__ __forceinline__ void each(F f) {
  if constexpr (I < N) {
    f.template operator()<I>();
    each<N, I + 1>(f);
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

// The tiles of a product grouped by at most 64 experts, found by every wave on its own from
// the offsets: lane e holds expert e's rows (offsets made non-decreasing and cut at
// the rows) and the tiles up to its last.  The tiles of the rows before the first and
// after the last group, of no expert, follow.  Against a plan kernel before the product (us a call):
// 70 rows of 32 experts, 1504 x 2049, 14.1 against 16.4; 6007 rows, 2048 x 1408, 50.3 against 53.5.
struct OffsetTiles {
  int start, end, upto, experts;
  int before, after;           // rows of no expert: [0, before), [after, rows)
  int total;
};
__device__ __forceinline__ OffsetTiles scan_offsets(const MxGemm& p, int tile) {
  const int lane = threadIdx.x & 63;
  OffsetTiles s;
  s.start = lane < p.E ? min(max(p.offsets[lane], 0), p.rows) : 0;
  s.end = lane < p.E ? min(max(p.offsets[lane + 1], 0), p.rows) : 0;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) s.start = max(s.start, __shfl_up(s.start, d));   // (lanes below d: their own)
  s.end = lane < p.E ? max(s.end, s.start) : s.start;
  s.upto = lane < p.E ? (s.end - s.start + tile - 1) / tile : 0;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(s.upto, d);
    s.upto += lane >= d ? o : 0;
  }
  s.experts = __builtin_amdgcn_readlane(s.upto, 63);
  s.before = __builtin_amdgcn_readlane(s.start, 0);
  s.after = __builtin_amdgcn_readlane(s.end, p.E - 1);
  s.total = s.experts + (s.before + tile - 1) / tile + (p.rows - s.after + tile - 1) / tile;
  return s;
}
__device__ __forceinline__ RowTile offset_tile(const OffsetTiles& s, int rows, int tile, int tm) {
  if (tm < s.experts) {
    const int e = __builtin_ctzll(__ballot(s.upto > tm));
    const int start = __builtin_amdgcn_readlane(s.start, e), end = __builtin_amdgcn_readlane(s.end, e);
    const int own = (end - start + tile - 1) / tile, in = tm - (__builtin_amdgcn_readlane(s.upto, e) - own);
    return RowTile{e, start + in * tile, min(tile, end - start - in * tile), 0};
  }
  tm -= s.experts;
  const int before = (s.before + tile - 1) / tile;
  if (tm < before) return RowTile{-1, tm * tile, min(tile, s.before - tm * tile), 0};
  const int first = s.after + (tm - before) * tile;
  return RowTile{-1, first, min(tile, rows - first), 0};
}

// Sixteen rows of NT column tiles from a wave's accumulators (v[j]: lane 16 h + r has
// columns 16 j + 4 h .. + 3 of row r) to memory, through the wave's own stretch
// of LDS, so that a row leaves as whole lines: 16-byte stores of eight outputs (float32: two
// stores), or one output per lane where the rows are not aligned for that.
// row_at(i): the output row of the tile's row i; rows: how many there are.
constexpr int flush_floats(int nt) { return 16 * (16 * nt + 4); }
template <int NT, class Spec, class RowAt>
__device__ __forceinline__ void drain16(const Spec& p, const float* buf, int rows, int col0, RowAt row_at) {
  constexpr int COLS = 16 * NT, LD = COLS + 4, UNITS = COLS / 8;
  const int lane = threadIdx.x & 63;
  if (p.vec == 2) {
#pragma unroll
    for (int i = 0; i < (16 * UNITS + 63) / 64; ++i) {
      const int u = i * 64 + lane, lr = u / UNITS, c = (u % UNITS) * 8, col = col0 + c;
      if (u >= 16 * UNITS || lr >= rows || col >= p.N) continue;
      const f32x4 a = *(const f32x4*)(buf + lr * LD + c), b = *(const f32x4*)(buf + lr * LD + c + 4);
      float f[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
      const int64_t at = row_at(lr) * p.stride() + col;
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
#pragma unroll 4
    for (int i = 0; i < COLS / 4; ++i) {
      const int u = i * 64 + lane, lr = u / COLS, c = u % COLS, col = col0 + c;
      if (lr >= rows || col >= p.N) continue;
      float f = buf[lr * LD + c];
      const int64_t at = row_at(lr) * p.stride() + col;
      p.add_one(f, at);
      if (p.out_type == kTypeF32) ((float*)p.out)[at] = f;
      else ((uint16_t*)p.out)[at] = to_16(f, p.out_type);
      if (p.low_plane()) p.low_plane()[at] = f32_to_bf16(bf16_rest(f));
    }
  }
}

template <int NT, class Spec, class RowAt>
__device__ __forceinline__ void flush16(const Spec& p, float* buf, const f32x4* v, int rows, int col0, RowAt row_at) {
  constexpr int LD = 16 * NT + 4;
  const int lane = threadIdx.x & 63, r = lane & 15, h = lane >> 4;
  asm volatile("" ::: "memory");               // a wave's LDS accesses keep their order
#pragma unroll
  for (int j = 0; j < NT; ++j) *(f32x4*)(buf + r * LD + 16 * j + 4 * h) = v[j];
  asm volatile("" ::: "memory");
  drain16<NT>(p, buf, rows, col0, row_at);
}

// Rows 16 q .. of 32 x 32 accumulators v[0 .. WF): lane 32 h + r has columns
// 32 j + 8 e + 4 h .. + 3 of row r in elements 4 e .. 4 e + 3.
template <int NT, int WF, class Spec, class RowAt>
__device__ __forceinline__ void flush_half(const Spec& p, float* buf, const f32x16* v, int q, int rows, int col0,
                                           RowAt row_at) {
  constexpr int LD = 16 * NT + 4;
  const int lane = threadIdx.x & 63, r = lane & 31, h = lane >> 5;
  asm volatile("" ::: "memory");
  if ((r >> 4) == q) {
#pragma unroll
    for (int j = 0; j < WF; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        *(f32x4*)(buf + (r & 15) * LD + 32 * j + 8 * e + 4 * h) =
            (f32x4){v[j][4 * e], v[j][4 * e + 1], v[j][4 * e + 2], v[j][4 * e + 3]};
  }
  asm volatile("" ::: "memory");
  drain16<NT>(p, buf, rows, col0, row_at);
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
//
// Measured: 70 float16 rows of 32 experts, 1504 x 2049 (53 MB): 10.4 us with the weights in the last-level
// cache (5.1 TB/s), 15.6 from memory.  16 tokens, 8 of 64 experts: gate and up 2048 x 1024 37 us (123 MB,
// 3.3 TB/s), down 22; at 2080 x 1056, where rows are no power of two of
// bytes apart, 28 and 17 (4.7 TB/s).  16 x 5632 x 2048: 9.9 us, the chain of load, MFMA and join.

// Row tiles whose partial sums meet in LDS at once, and the f32x4 of LDS that this takes.
constexpr int few_pass(int rt, int nw, int w) {
  int rp = rt;
  while (rp > 1 && w * rp * nw > 32) rp /= 2;
  return rp;
}
constexpr int few_lds(int rt, int nw, int w) {
  const int rp = few_pass(rt, nw, w);
  return (rp < rt ? 2 : 1) * w * rp * nw * 64;
}

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
    const bool gather = p.xperm;
    const uint16_t* xb = gather ? p.x : p.x + (int64_t)first * p.K;
    const uint32_t xbytes = (uint32_t)((int64_t)(gather ? p.xrows : rows) * p.K * 2);
    __amdgpu_buffer_rsrc_t xr[NL];
#pragma unroll
    for (int q = 0; q < NL; ++q) xr[q] = buffer(xb + q * p.plane, xbytes);
    uint32_t xoff[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int lr = 16 * i + r;
      const int xrow = lr >= rows ? 0 : p.xperm ? p.xperm[first + lr] / p.xdiv : lr;
      xoff[i] = lr >= rows ? kNowhere : (uint32_t)xrow * (uint32_t)p.K * 2u + h * 64;
    }
    const int kb = p.K / 32, chunks = (kb + 3) / 4;
    const int64_t wrow = (int64_t)expert * p.wrows + n0;
    const int cols = p.N - n0;
    const int wbytes = min(cols, 16 * CT) * (p.K / 2);
    const __amdgpu_buffer_rsrc_t wr[2] = {buffer(p.w + wrow * (p.K / 8), wbytes),
                                          buffer((FUSED ? p.w2 : p.w) + wrow * (p.K / 8), wbytes)};
    const __amdgpu_buffer_rsrc_t sr[2] = {buffer(p.s + wrow * kb, wbytes / 16),
                                          buffer((FUSED ? p.s2 : p.s) + wrow * kb, wbytes / 16)};

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
          w[u][j] = load16(wr[j / CT], in ? (uint32_t)col * (uint32_t)(p.K / 2) + c * 64 + h * 16 : kNowhere);
          s[u][j] = load1(sr[j / CT], in ? (uint32_t)(col * kb + 4 * c + h) : kNowhere);
        }
#pragma unroll
        for (int q = 0; q < NL; ++q)
#pragma unroll
          for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              x[u][q][i][k] = load16(xr[q], in && xoff[i] != kNowhere ? xoff[i] + c * 256 + k * 16 : kNowhere);
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

  // the waves' sums, RP row tiles at a time: [wave][i][j][lane], added in wave order
  constexpr int RP = few_pass(RT, NW, W), PASS = W * RP * NW * 64;
#pragma unroll
  for (int i0 = 0; i0 < RT; i0 += RP) {
    f32x4* part = lds + (i0 / RP & 1) * PASS;   // two stretches in turn: one barrier a pass
#pragma unroll
    for (int i = 0; i < RP; ++i)
#pragma unroll
      for (int j = 0; j < NW; ++j) part[((wave * RP + i) * NW + j) * 64 + lane] = acc[i0 + i][j];
    __syncthreads();
    for (int f = wave; f < RP * CT; f += W) {
      const int i = f / CT, j = f % CT;
      f32x4 g = {0.0f, 0.0f, 0.0f, 0.0f}, u = g;
#pragma unroll
      for (int v = 0; v < W; ++v) {
        g += part[((v * RP + i) * NW + j) * 64 + lane];
        if constexpr (FUSED) u += part[((v * RP + i) * NW + j + CT) * 64 + lane];
      }
      if constexpr (FUSED) {
#pragma unroll
        for (int e = 0; e < 4; ++e) g[e] = silu_times(g[e], u[e]);
      }
      const int lr = 16 * (i0 + i) + r;
      if (lr < rows) {
        const int row = p.perm ? p.perm[first + lr] : first + lr;
        finish4(p, (int64_t)row * p.N, n0 + 16 * j + 4 * h, g);
      }
    }
  }
}

// Rows of the block: a tile of the table, or of a dense product.
template <int RT, int CT, int XS, bool FUSED, int W, int U>
__global__ __launch_bounds__(64 * W, 2) void mx4_few_kernel(MxGemm p) {
  __shared__ f32x4 lds[few_lds(RT, FUSED ? 2 * CT : CT, W)];
#ifdef SWQ_LDS_POISON
  lds_poison(lds, sizeof(lds), kPoisonFloat);
  __syncthreads();
#endif
  const int ntn = (p.N + 16 * CT - 1) / (16 * CT);
  int tm = blockIdx.x / ntn;
  const int tn = blockIdx.x - tm * ntn;
  int expert = 0, first = tm * 16 * RT, rows = min(16 * RT, p.rows - first);
  if (p.offsets) {
    const OffsetTiles s = scan_offsets(p, 16 * RT);
    if (tm >= s.total) return;
    const RowTile t = offset_tile(s, p.rows, 16 * RT, tm);
    expert = t.expert, first = t.first, rows = t.rows;
  } else if (p.tiles) {
    if (tm >= *p.ntiles) return;
    const RowTile t = p.tiles[tm];
    expert = t.expert, first = t.first, rows = t.rows;
  }
  expert = __builtin_amdgcn_readfirstlane(expert);
  first = __builtin_amdgcn_readfirstlane(first);
  rows = __builtin_amdgcn_readfirstlane(rows);
  few_rows<RT, CT, XS, FUSED, W, U>(p, expert, first, rows, tn * 16 * CT, lds);
}

// ----------------------------------------------------------- one-row kernels ----
//
// One row of x: the weights' bytes are all there is.  A wave takes U chunks at once; its
// part of x is one load of 16 bytes per lane, put into the wave's own stretch of
// LDS and read back by every column of the operand (all 16 rows of the MFMA's second
// operand hold the same row; row 0's result counts).  A lane's four loads of codes are neighbours, so
// a wave takes whole lines of the weights.
//
// Bound by latency (the launch, x, the weights, the join) where a CU has one block: 2048 x 5632
// 5.0 us (6.1 MB).  One token, 8 of 64 experts, 2048 x 1024: gate and up 9.0 us (17.8 MB, 2.0 TB/s),
// down with the weighted sum 7.4.

constexpr int kRowU = 4, kRowStretch = kRowU * 16;       // chunks in flight; u32x4 of LDS per wave and plane

// Sums of a wave over the chunks 4 i .. 4 i + 3, i = first, first + step, ..., for the 16 columns
// of each of NW matrices (four neighbours: 256 bytes of each row).
template <int XS, int NW>
__device__ __forceinline__ void row_sums(const __amdgpu_buffer_rsrc_t (&wr)[NW], const __amdgpu_buffer_rsrc_t (&sr)[NW],
                                         const uint16_t* x, int64_t plane, int K, int first, int step, u32x4* own,
                                         f32x4 (&acc)[NW]) {
  constexpr int NP = XS == kXBf16 ? 1 : 2, NL = XS == kXPlanes ? 2 : 1;
  const int lane = threadIdx.x & 63, r = lane & 15, h = lane >> 4;
  const int kb = K / 32, chunks = (kb + 3) / 4;
  __amdgpu_buffer_rsrc_t xr[NL];
#pragma unroll
  for (int q = 0; q < NL; ++q) xr[q] = buffer(x + q * plane, K * 2);
  const uint32_t woff = (uint32_t)r * (uint32_t)(K / 2) + h * 16, soff = (uint32_t)(r * kb + h);
  for (int c0 = first * kRowU; c0 < chunks; c0 += step * kRowU) {
    u32x4 w[kRowU][NW], xv[NL];
    uint32_t s[kRowU][NW];
#pragma unroll
    for (int u = 0; u < kRowU; ++u) {
      const int c = c0 + u;
      const bool in = 4 * c + h < kb;
#pragma unroll
      for (int j = 0; j < NW; ++j) {
        w[u][j] = load16(wr[j], in ? woff + c * 64 : kNowhere);
        s[u][j] = load1(sr[j], in ? soff + 4 * c : kNowhere);
      }
    }
    // lane 16 u + p: the 16 bytes p of chunk u (past K: zeros, by the descriptor's end)
#pragma unroll
    for (int q = 0; q < NL; ++q) xv[q] = load16(xr[q], (uint32_t)c0 * 256u + lane * 16);
    __builtin_amdgcn_sched_barrier(0);         // every load is out before the first is waited for
    asm volatile("" ::: "memory");             // a wave's LDS accesses keep their order
    if constexpr (XS == kXF16) {
      bf16x8 hi, lo;
      split_f16x8(__builtin_bit_cast(f16x8, xv[0]), hi, lo);
      own[lane] = __builtin_bit_cast(u32x4, hi);
      own[kRowStretch + lane] = __builtin_bit_cast(u32x4, lo);
    } else {
#pragma unroll
      for (int q = 0; q < NL; ++q) own[q * kRowStretch + lane] = xv[q];
    }
    asm volatile("" ::: "memory");
#pragma unroll
    for (int u = 0; u < kRowU; ++u)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        bf16x8 b[NP];
#pragma unroll
        for (int q = 0; q < NP; ++q) b[q] = __builtin_bit_cast(bf16x8, own[q * kRowStretch + 16 * u + 4 * h + k]);
#pragma unroll
        for (int j = 0; j < NW; ++j) {
          const bf16x8 a = mx4_word(w[u][j][k], e8m0_operand(s[u][j]));
#pragma unroll
          for (int q = 0; q < NP; ++q) acc[j] = mfma_bf16(a, b[q], acc[j]);
        }
      }
  }
}

// 16 columns (SwiGLU: of both matrices) of one row per block: a dense product's row, or the slot
// of p.ids.  The W waves' sums are added in wave order.
template <int XS, bool FUSED, int W>
__global__ __launch_bounds__(64 * W) void mx4_row_kernel(MxGemm p) {
  constexpr int NW = FUSED ? 2 : 1, NP = XS == kXBf16 ? 1 : 2;
  __shared__ u32x4 xs[W * NP * kRowStretch];
  __shared__ f32x4 part[W * NW * 4];
#ifdef SWQ_LDS_POISON
  lds_poison(xs, sizeof(xs), kPoisonFloat);
  lds_poison(part, sizeof(part), kPoisonFloat);
  __syncthreads();
#endif
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, h = lane >> 4;
  const int ntn = (p.N + 15) / 16;
  const int slot = blockIdx.x / ntn, n0 = (blockIdx.x - slot * ntn) * 16;
  const int expert = p.ids ? __builtin_amdgcn_readfirstlane(p.ids[slot]) : 0;
  if (expert < 0 || expert >= p.E) return;     // a skipped slot: nothing reads its row
  const int kb = p.K / 32, cols = min(16, p.N - n0);
  const int64_t wrow = (int64_t)expert * p.wrows + n0;
  __amdgpu_buffer_rsrc_t wr[NW], sr[NW];
#pragma unroll
  for (int j = 0; j < NW; ++j) {
    wr[j] = buffer((j ? p.w2 : p.w) + wrow * (p.K / 8), cols * (p.K / 2));
    sr[j] = buffer((j ? p.s2 : p.s) + wrow * kb, cols * kb);
  }
  f32x4 acc[NW];
#pragma unroll
  for (int j = 0; j < NW; ++j) acc[j] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
  row_sums<XS, NW>(wr, sr, p.x + (int64_t)(slot / p.xdiv) * p.K, p.plane, p.K, wave, W, xs + wave * NP * kRowStretch,
                   acc);
  if (r == 0) {
#pragma unroll
    for (int j = 0; j < NW; ++j) part[(wave * NW + j) * 4 + h] = acc[j];
  }
  __syncthreads();
  if (wave == 0 && r == 0) {
    f32x4 g[NW];
#pragma unroll
    for (int j = 0; j < NW; ++j) {
      g[j] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int v = 0; v < W; ++v) g[j] += part[(v * NW + j) * 4 + h];
    }
    if constexpr (FUSED) {
#pragma unroll
      for (int e = 0; e < 4; ++e) g[0][e] = silu_times(g[0][e], g[1][e]);
    }
    finish4(p, (int64_t)slot * p.N, n0 + 4 * h, g[0]);
  }
}

// The experts' down projection of few tokens with the weighted sum: block (token, 16
// columns).  `share` waves (a power of two) take a slot together, the W / share
// teams take the token's slots in turn, and the waves' sums, times the slots' weights,
// are added in wave order.
template <int XS, int W>
__global__ __launch_bounds__(64 * W) void mx4_down_kernel(MxGemm p, const float* __restrict__ weights, int k,
                                                          int share) {
  constexpr int NP = XS == kXBf16 ? 1 : 2;
  __shared__ u32x4 xs[W * NP * kRowStretch];
  __shared__ f32x4 part[W * 4];
#ifdef SWQ_LDS_POISON
  lds_poison(xs, sizeof(xs), kPoisonFloat);
  lds_poison(part, sizeof(part), kPoisonFloat);
  __syncthreads();
#endif
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, h = lane >> 4;
  const int ntn = (p.N + 15) / 16;
  const int t = blockIdx.x / ntn, n0 = (blockIdx.x - t * ntn) * 16;
  const int kb = p.K / 32, cols = min(16, p.N - n0);
  f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int j = wave / share; j < k; j += W / share) {
    const int slot = t * k + j;
    const int expert = __builtin_amdgcn_readfirstlane(p.ids[slot]);
    if (expert < 0 || expert >= p.E) continue;
    const float wt = weights[slot];
    const int64_t wrow = (int64_t)expert * p.wrows + n0;
    const __amdgpu_buffer_rsrc_t wr[1] = {buffer(p.w + wrow * (p.K / 8), cols * (p.K / 2))};
    const __amdgpu_buffer_rsrc_t sr[1] = {buffer(p.s + wrow * kb, cols * kb)};
    f32x4 acc[1] = {{0.0f, 0.0f, 0.0f, 0.0f}};
    row_sums<XS, 1>(wr, sr, p.x + (int64_t)slot * p.K, p.plane, p.K, wave % share, share, xs + wave * NP * kRowStretch,
                    acc);
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[e] = fmaf(wt, acc[0][e], sum[e]);
  }
  if (r == 0) part[wave * 4 + h] = sum;
  __syncthreads();
  if (wave == 0 && r == 0) {
    f32x4 y = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int v = 0; v < W; ++v) y += part[v * 4 + h];
    finish4(p, (int64_t)t * p.N, n0 + 4 * h, y);
  }
}

// ------------------------------------------------------------ tiled kernel ----
//
// WM x WN waves, each MF x NF accumulators of 16 x 16 over 16 MF rows of x and
// 16 NF columns of W (SwiGLU: NF / 2 column tiles of the gate and the same of the
// up matrix).  A chunk is 128 inputs: lane 16 h + r takes block h of a chunk
// in four steps, so its codes are one 16-byte load and its scale one byte,
// straight from memory to registers S - 1 chunks ahead (a column's codes are used
// by WM waves only).  x goes through LDS, [BM * NP][128] bf16, S buffers, by
// loads that write LDS; 16-byte unit u of a row sits at u ^ (row & 15), which keeps the
// 64-byte pieces that four lanes load whole.  (Two rows of a read still meet in a bank, 4 cycles a read.
// A placement without that, in whole pieces, took the same time; one that breaks the pieces
// 294 us where this takes 225: the loads, not the reads, count.)
//
// Measured: 2048 x 4096 x 14336 225 us, 1.07 PFLOP/s (the library's bf16 product of that shape 205);
// matrix units 54 % busy at the 1.9 GHz that the card's power leaves.  8192 x 2560 x 10240 379 us,
// 1.13 PFLOP/s.  32768 rows of 64 experts: gate and up 2048 x 1024 303 us, 0.91 PFLOP/s, down 2 x 99 us, 0.70: a ninth
// of the tiles' rows is past the experts' ends, the last round of tiles leaves CUs idle, and the
// down projection's short K ends in 128 KB of float32 per tile.  Float16 x, two operands: 2048 x
// 4096 x 14336 421 to 463 us, 1.04 to 1.14 PFLOP/s of bf16 products.
template <int MF, int NF, int WM, int WN, int NP, int S, bool FUSED, bool SPLIT>
__global__ __launch_bounds__(64 * WM * WN, 2) void mx4_gemm_kernel(MxGemm p) {
  constexpr int W = WM * WN, BM = 16 * MF * WM, ROWS = BM * NP, BN = 16 * NF * WN, BNO = FUSED ? BN / 2 : BN;
  constexpr int DMA = ROWS / (4 * W);           // loads per lane and chunk, four rows each per wave
  static_assert(ROWS % (4 * W) == 0 && W % 4 == 0 && (!FUSED || NF % 2 == 0));
  __shared__ __attribute__((aligned(1024))) char lds[S * ROWS * 256];
#ifdef SWQ_LDS_POISON
  lds_poison(lds, sizeof(lds), kPoisonFloat);
  __syncthreads();
#endif
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, h = lane >> 4;
  const int wm = wave / WN, wn = wave % WN;

  const int ntn = (p.N + BNO - 1) / BNO;
  int tm, tn, ntm = (p.rows + BM - 1) / BM;
  OffsetTiles ot;
  if (p.offsets) {
    ot = scan_offsets(p, BM);
    ntm = ot.total;
  } else if (p.tiles) {
    ntm = *p.ntiles;
  }
  if (!tile_of(blockIdx.x, ntm, ntn, tm, tn)) return;
  const int split = SPLIT ? blockIdx.y : 0;     // of K: its share of the chunks, its part of the partial sums
  int expert = 0, first = tm * BM, rows = min(BM, p.rows - first);
  if (p.offsets || p.tiles) {
    const RowTile t = p.offsets ? offset_tile(ot, p.rows, BM, tm) : p.tiles[tm];
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

  const int c_begin = SPLIT ? split * p.split_chunks : 0;
  const int chunks = SPLIT ? min((p.K + 127) / 128, c_begin + p.split_chunks) : (p.K + 127) / 128;
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
    // load i of chunk c (past K: zeros)
    const auto load_x = [&]<int i>(int c, int buf) SWQ_INLINE {
      dma16(xr[(i * 4 * W) / BM],
            __builtin_amdgcn_readfirstlane(lds_addr(lds) + buf * (ROWS * 256) + (i * 4 * W + wave * 4) * 256),
            (!SPLIT || c < chunks) && c * 128 + du * 8 < p.K ? xoff[i] + (uint32_t)c * 256u : kNowhere);
    };

    // W: the columns of this wave; rows past N read zeros
    const int kb = p.K / 32;
    const int64_t wrow = (int64_t)expert * p.wrows + n0;
    const int wn_rows = p.N - n0;
    uint32_t woff[NF], soff[NF];
#pragma unroll
    for (int j = 0; j < NF; ++j) {
      const int col = FUSED ? 16 * (wn * (NF / 2) + j % (NF / 2)) + r : 16 * (wn * NF + j) + r;
      woff[j] = (uint32_t)col * (uint32_t)(p.K / 2) + h * 16;
      soff[j] = (uint32_t)col * (uint32_t)kb + h;
    }
    const __amdgpu_buffer_rsrc_t wr0 = buffer(p.w + wrow * (p.K / 8), min(wn_rows, BNO) * (p.K / 2));
    const __amdgpu_buffer_rsrc_t wr1 =
        buffer((FUSED ? p.w2 : p.w) + wrow * (p.K / 8), min(wn_rows, BNO) * (p.K / 2));
    const __amdgpu_buffer_rsrc_t sr0 = buffer(p.s + wrow * kb, min(wn_rows, BNO) * kb);
    const __amdgpu_buffer_rsrc_t sr1 = buffer((FUSED ? p.s2 : p.s) + wrow * kb, min(wn_rows, BNO) * kb);
    // S stages: a chunk's x in LDS, its codes and scales in registers, loaded S - 1 chunks ahead
    u32x4 wc[S][NF];
    uint32_t sc[S][NF];
    const auto load_w = [&]<int b, int j>(int c) SWQ_INLINE {
      constexpr bool up = FUSED && j >= NF / 2;
      const bool in = (!SPLIT || c < chunks) && 4 * c + h < kb;
      wc[b][j] = load16(up ? wr1 : wr0, in ? woff[j] + c * 64 : kNowhere);
      sc[b][j] = load1(up ? sr1 : sr0, in ? soff[j] + 4 * c : kNowhere);
    };
    constexpr int LOADS = 2 * NF + DMA;
    each<S - 1>([&]<int b>() SWQ_INLINE {
      each<NF>([&]<int j>() SWQ_INLINE { load_w.template operator()<b, j>(c_begin + b); });
      each<DMA>([&]<int i>() SWQ_INLINE { load_x.template operator()<i>(c_begin + b, b); });
      __builtin_amdgcn_sched_barrier(0);        // the waits below count on the loads' order
    });

    // Chunk c, in stage b; loads past the last chunk read nothing, chunks past it add zeros.
    const auto chunk = [&]<int b>(int c) SWQ_INLINE {
      wait_vmcnt<(S - 2) * LOADS>();            // the later chunks' loads may still be out
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      // The chunk's operands of x one after another (step, plane, row tile), each read two ahead of its
      // MFMAs.  What else there is to do -- the loads of chunk c + S - 1, the conversion of the
      // next step's weights -- stands one piece at a time between MFMAs, in whose
      // cycles it hides.
      constexpr int PER = MF * NP, ALL = 4 * PER, GAP = PER / 4, ahead = (b + S - 1) % S;
      const char* xt = lds + b * (ROWS * 256) + (wm * MF * 16 + r) * 256;
      bf16x8 x[3];
      u32x4 w[2][NF];
      const auto read_x = [&]<int n>() SWQ_INLINE {
        constexpr int step = n / PER, q = n % PER / MF, i = n % MF;
        x[n % 3] = *(const bf16x8*)(xt + (((4 * h + step) ^ r) * 16) + (q * BM + 16 * i) * 256);
      };
      read_x.template operator()<0>();
      read_x.template operator()<1>();
#pragma unroll
      for (int j = 0; j < NF; ++j) w[0][j] = __builtin_bit_cast(u32x4, mx4_word(wc[b][j][0], e8m0_operand(sc[b][j])));
      each<ALL * NF>([&]<int m>() SWQ_INLINE {
        constexpr int n = m / NF, j = m % NF, step = n / PER, i = n % MF, l = m % (PER * NF);
        if constexpr (j == 0 && n + 2 < ALL) read_x.template operator()<n + 2>();
        if constexpr (m % 2 == 1 && m / 2 < NF) load_w.template operator()<ahead, m / 2>(c + S - 1);
        if constexpr (m % 2 == 1 && m / 2 >= NF && m / 2 < NF + DMA)
          load_x.template operator()<m / 2 - NF>(c + S - 1, ahead);
        if constexpr (step < 3 && l % GAP == GAP - 1) {
          constexpr int k = l / GAP, jj = k / 4, e = k % 4;
          w[(step + 1) & 1][jj][e] = mx4_pair<e>(wc[b][jj][step + 1], e8m0_operand(sc[b][jj]));
        }
        acc[i][j] = mfma_bf16(__builtin_bit_cast(bf16x8, w[step & 1][j]), x[n % 3], acc[i][j]);
        __builtin_amdgcn_sched_barrier(0);
      });
    };
    for (int c = c_begin; c < chunks; c += S)
      each<S>([&]<int b>() SWQ_INLINE { chunk.template operator()<b>(c + b); });
    wait_vmcnt<0>();           // no load past the end may still write LDS
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
      return (int64_t)(p.perm ? p.perm[slot] : slot) + (int64_t)split * p.rows;
    });
  }
}

// The sums of a K split, added in the order of the splits: four neighbouring outputs per thread.
// 256 x 5632 x 2048: 4 us after the 16 of the split tiles, a launch and a load's latency.
__global__ __launch_bounds__(256) void mx4_join_kernel(MxGemm p) {
  const int per = (p.N + 3) / 4;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, row = i / per;
  const int n = (int)(i - row * per) * 4;
  if (row >= p.rows) return;
  const float* part = (const float*)p.parts + row * p.N + n;
  const int64_t step = (int64_t)p.rows * p.N;
  f32x4 y = {0.0f, 0.0f, 0.0f, 0.0f};
  if (p.N % 4 == 0) {
    for (int s = 0; s < p.splits; ++s) y += *(const f32x4*)(part + s * step);
  } else {
    for (int s = 0; s < p.splits; ++s)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (n + e < p.N) y[e] += part[s * step + e];
  }
  finish4(p, row * p.N, n, y);
}

// ----------------------------------------------------- two MXFP4 operands ----
//
// 32 x 32 x 64 scaled MFMA: lane 32 h + r holds row r's block h of a k-step of 64
// inputs, 32 codes in four registers, and the byte of its scale operand that
// the k-step selects.  (The 16 x 16 x 128 form is held to 27 cycles where
// its rate would be 16 -- 5.6 PFLOP/s on registers alone, zeros or not; this
// one reaches 9.7 PFLOP/s on zeros and 6.4 on random codes, the card's power
// limit.)
//
// The scales' bytes lie K / 32 apart, at any address, and a stage of 128
// inputs needs four per row.  A first kernel lays them out as the MFMA takes
// them: for 32 rows and a stage, two bytes per lane, byte e for k-step e
// (blocks past K: 0).  8192 + 10240 rows of 80: 5 us, 1.5 MB in and out, latency.
__global__ __launch_bounds__(256) void mx4_scale_kernel(const uint8_t* __restrict__ sa, int M,
                                                        const uint8_t* __restrict__ sw, int N, int kb, int stages,
                                                        int pad_a, int pad_w, uint16_t* __restrict__ out) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;      // [32 rows][stage][row]
  const int64_t group = i / (32 * stages);
  const int t = (int)((i - group * 32 * stages) >> 5), row = (int)group * 32 + (int)(i & 31);
  if (row >= pad_a + pad_w) return;
  const bool is_a = row < pad_a;
  const int at = is_a ? row : row - pad_a;
  const uint8_t* s = (is_a ? sa : sw) + (int64_t)at * kb;
  const bool live = at < (is_a ? M : N);
  uint32_t b[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) b[e] = live && 4 * t + e < kb ? s[4 * t + e] : 0u;
  uint16_t* o = out + (group * stages + t) * 64 + (row & 31);
  o[0] = (uint16_t)(b[0] | b[2] << 8);
  o[32] = (uint16_t)(b[1] | b[3] << 8);
}

template <int E>
__device__ __forceinline__ f32x16 mfma_mx4_wide(u32x4 a, uint32_t sa, u32x4 b, uint32_t sb, f32x16 c) {
  const i32x8 A = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i32x8 B = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(A, B, c, 4, 4, E, (int)sa, E, (int)sb);
}

// As dma16, four bytes per lane.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void dma4(i32x4 rs, uint32_t lds_base, uint32_t voff) {
  asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dword %1, %2, 0 offen lds"
               ::"s"(lds_base), "v"(voff), "s"(rs) : "memory", "m0");
}
#pragma clang diagnostic pop

// A wave's 32 x 32 accumulators to aligned rows: lane 32 h + r has columns 8 e + 4 h .. + 3
// of row r in elements 4 e ..; for 16-bit outputs the halves of the wave swap
// pieces of two such quads, so that every lane stores eight neighbours.
template <int TYPE, int AF, int WF>
__device__ __forceinline__ void store_wide(const Mx4Matmul& p, const f32x16 (&acc)[AF][WF], int mw, int nw) {
  const int lane = threadIdx.x & 63, r = lane & 31, h = lane >> 5;
#pragma unroll
  for (int i = 0; i < AF; ++i) {
    const int m = mw + 32 * i + r;
    if (m >= p.M) continue;
    const int64_t at = (int64_t)m * p.ld;
#pragma unroll
    for (int j = 0; j < WF; ++j) {
      const f32x16& v = acc[i][j];
      if constexpr (TYPE == kTypeF32) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int col = nw + 32 * j + 8 * e + 4 * h;
          if (col < p.N)
            *(f32x4*)((float*)p.out + at + col) = (f32x4){v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]};
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
          uint32_t q[4];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t x = pack16<TYPE>(v[4 * e + 2 * k], v[4 * e + 2 * k + 1]);
            const uint32_t y = pack16<TYPE>(v[4 * e + 4 + 2 * k], v[4 * e + 5 + 2 * k]);
            const auto sw = __builtin_amdgcn_permlane32_swap(x, y, false, false);
            q[k] = sw[0];
            q[2 + k] = sw[1];
          }
          const int col = nw + 32 * j + 8 * (e + h);
          if (col < p.N) *(u32x4*)((uint16_t*)p.out + at + col) = (u32x4){q[0], q[1], q[2], q[3]};
        }
      }
    }
  }
}

// WM x WN waves of 32 AF x 32 WF outputs.  A stage is 128 inputs, 64 bytes a row
// of each operand and its scales, S stages in LDS; a k-step reads its successor's
// operands into registers while its MFMAs run, and a stage that has been read makes
// room for the loads of the one S ahead.  16-byte unit u of a row sits at u ^ (row / 4 & 3):
// the rows that a read touches lie in different banks (no conflict cycles counted).  As many blocks as
// the CUs hold take the tiles in turn, and a block's next loads go out before its stores.
//
// 8192 x 2560 x 10240: 131 to 134 us, 3.3 PFLOP/s, 168 MB of outputs; matrix units 45 % busy.  What bounds it was not
// found: its reads from L2 (13.1 M requests of 64 bytes, 840 MB, 86 % of all requests hit) come to 6.4 TB/s, less than
// the 8.3 that the product of bf16 rows takes, and waves wait 46 % of their cycles; the outputs, 32 us of the
// memory's time, overlap only in part.
template <int AF, int WF, int WM, int WN, int S>
struct MmShape {
  static constexpr int W = WM * WN, BM = 32 * AF * WM, BN = 32 * WF * WN, ROWS = BM + BN;
  // of one wave and stage: loads of 16 rows of codes, loads of the scales of 64 rows
  static constexpr int LOADS = ROWS / (16 * W), SCALES = (ROWS / 64 + W - 1) / W, PER = LOADS + SCALES;
  static constexpr int CODES = ROWS * 64, STAGE = CODES + SCALES * W * 256, LDS = S * STAGE;
  static_assert(ROWS % (16 * W) == 0 && BM % (16 * W) == 0 && BM % 64 == 0);
};

template <int AF, int WF, int WM, int WN, int S, int OCC>
__global__ __launch_bounds__(64 * WM * WN, OCC * WM * WN / 4) void mx4_matmul_kernel(
    Mx4Matmul p, const uint16_t* __restrict__ scales, int stages, int pad_a) {
  using Sh = MmShape<AF, WF, WM, WN, S>;
  constexpr int BM = Sh::BM, BN = Sh::BN, W = Sh::W;
  __shared__ __attribute__((aligned(1024))) char lds[Sh::LDS];
#ifdef SWQ_LDS_POISON
  lds_poison(lds, sizeof(lds), kPoisonFloat);
  __syncthreads();
#endif
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 31, h = lane >> 5;
  const int wm = wave / WN, wn = wave % WN;
  const int ntm = (p.M + BM - 1) / BM, ntn = (p.N + BN - 1) / BN, row_bytes = p.K / 2;
  const int unit = (lane & 3) ^ (lane >> 4);           // (row / 4 & 3) == lane / 16

  // One tile's loads.  Codes: load i of wave w takes rows 16 (W i + w) + lane / 4 of the two operands put
  // together, a row past the end repeating the tile's first.  Scales: load i of wave w
  // takes the 128 bytes of row groups 2 (W i + w) and the next (the operands put together).
  constexpr int OF_A = BM / (16 * W);                  // the loads that are of A
  // The descriptors cover the whole operands of the launch (under 4 GiB each, kSlabBytes): they stay in
  // scalar registers whatever the tile.
  const i32x4 ra = make_srsrc(p.a, (uint32_t)p.M * (uint32_t)row_bytes);
  const i32x4 rw = make_srsrc(p.w, (uint32_t)p.N * (uint32_t)row_bytes);
  const i32x4 rs = make_srsrc(scales, (uint32_t)(pad_a + ntn * BN) * (uint32_t)stages * 4u);
  int m0 = 0, n0 = 0;
  uint32_t off[Sh::LOADS], soff[Sh::SCALES];
  const auto aim = [&](int block) SWQ_INLINE {
    int tm, tn;
    if (!tile_of(block, ntm, ntn, tm, tn)) return false;
    m0 = tm * BM, n0 = tn * BN;
#pragma unroll
    for (int i = 0; i < Sh::LOADS; ++i) {
      const int row = 16 * (W * i + wave) + (lane >> 2);
      const int at = i < OF_A ? (m0 + row < p.M ? m0 + row : m0) : (n0 + row - BM < p.N ? n0 + row - BM : n0);
      off[i] = (uint32_t)at * (uint32_t)row_bytes + unit * 16;
    }
#pragma unroll
    for (int i = 0; i < Sh::SCALES; ++i) {
      const int grp = 2 * (W * i + wave) + h;
      const int at = grp < BM / 32 ? m0 / 32 + grp : (pad_a + n0) / 32 + grp - BM / 32;
      soff[i] = grp < Sh::ROWS / 32 ? (uint32_t)at * (uint32_t)stages * 128u + r * 4 : kNowhere;
    }
    return true;
  };
  const uint32_t lds0 = lds_addr(lds);
  // load i of a stage: codes, then scales
  const auto load = [&]<int i>(int t, int slot) SWQ_INLINE {
    const uint32_t base = lds0 + slot * Sh::STAGE;
    if constexpr (i < Sh::LOADS)
      dma16(i < OF_A ? ra : rw, __builtin_amdgcn_readfirstlane(base + (W * i + wave) * 1024),
            t * 128 + unit * 32 < p.K ? off[i] + (uint32_t)t * 64u : kNowhere);
    else
      dma4(rs, __builtin_amdgcn_readfirstlane(base + Sh::CODES + (W * (i - Sh::LOADS) + wave) * 256),
           t < stages && soff[i - Sh::LOADS] != kNowhere ? soff[i - Sh::LOADS] + (uint32_t)t * 128u : kNowhere);
  };

  f32x16 acc[AF][WF];
  u32x4 a[2][AF], w[2][WF];
  uint32_t sa[2][AF], sw[2][WF];
  // operand i of k-step k: first x's, then w's
  const auto read_code = [&]<int k, int i>(int slot) SWQ_INLINE {
    const char* s = lds + slot * Sh::STAGE + r * 64 + (((2 * k + h) ^ (r >> 2 & 3)) * 16);
    if constexpr (i < AF) a[k][i] = *(const u32x4*)(s + (wm * AF + i) * 2048);
    else w[k][i - AF] = *(const u32x4*)(s + BM * 64 + (wn * WF + i - AF) * 2048);
  };
  const auto read_scale = [&]<int set, int i>(int slot) SWQ_INLINE {
    const char* s = lds + slot * Sh::STAGE + Sh::CODES + lane * 2;
    if constexpr (i < AF) sa[set][i] = *(const uint16_t*)(s + (wm * AF + i) * 128);
    else sw[set][i - AF] = *(const uint16_t*)(s + (BM / 32 + wn * WF + i - AF) * 128);
  };
  const auto meet = [&]() SWQ_INLINE {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  // A k-step's MFMAs; before(n) is issued in front of the n-th, so that one LDS
  // read and one load at a time share its cycles.
  const auto products = [&]<int E, int SET>(auto before) SWQ_INLINE {
    each<AF * WF>([&]<int n>() SWQ_INLINE {
      constexpr int i = n / WF, j = n % WF;
      before.template operator()<n>();
      acc[i][j] = mfma_mx4_wide<E>(w[E][j], sw[SET][j], a[E][i], sa[SET][i], acc[i][j]);
      __builtin_amdgcn_sched_barrier(0);
    });
  };
  const auto begin = [&]() SWQ_INLINE {
    each<S>([&]<int t>() SWQ_INLINE { each<Sh::PER>([&]<int i>() SWQ_INLINE { load.template operator()<i>(t, t); }); });
  };
  // One stage.  Loads are issued past the last stage too (they read nothing),
  // so the counts hold to the end.
  constexpr int FRAGS = AF + WF, M = AF * WF;
  constexpr int READS = (FRAGS + M - 1) / M, ISSUES = (Sh::PER + M - 1) / M;
  int slot = 0;
  const auto one = [&]<int SET>(int t) SWQ_INLINE {
    products.template operator()<0, SET>([&]<int n>() SWQ_INLINE {
      each<READS>([&]<int e>() SWQ_INLINE {
        if constexpr (n * READS + e < FRAGS) read_code.template operator()<1, n * READS + e>(slot);
      });
    });
    wait_vmcnt<(S - 2) * Sh::PER>();           // stage t + 1 is there
    meet();
    const int was = slot;
    slot = slot + 1 == S ? 0 : slot + 1;
    products.template operator()<1, SET>([&]<int n>() SWQ_INLINE {
      each<READS>([&]<int e>() SWQ_INLINE {
        if constexpr (n * READS + e < FRAGS) {
          read_code.template operator()<0, n * READS + e>(slot);
          read_scale.template operator()<(SET ^ 1), n * READS + e>(slot);
        }
      });
      each<ISSUES>([&]<int e>() SWQ_INLINE {
        if constexpr (n * ISSUES + e < Sh::PER) load.template operator()<n * ISSUES + e>(t + S, was);
      });
    });
  };

  // The block's tiles, one after another: the next one's first loads are on their way
  // while this one's sums go out.
  int block = blockIdx.x;
  if (!aim(block)) return;
  begin();
  while (true) {
#pragma unroll
    for (int i = 0; i < AF; ++i)
#pragma unroll
      for (int j = 0; j < WF; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
    wait_vmcnt<(S - 1) * Sh::PER>();
    meet();
    slot = 0;
    each<FRAGS>([&]<int i>() SWQ_INLINE {
      read_code.template operator()<0, i>(0);
      read_scale.template operator()<0, i>(0);
    });
    for (int t = 0; t < stages; t += 2) {      // an odd count's last half adds zeros
      one.template operator()<0>(t);
      one.template operator()<1>(t + 1);
    }
    wait_vmcnt<0>();           // no load past the end may still write LDS
    meet();

    const int mw = m0 + wm * 32 * AF, nw = n0 + wn * 32 * WF;
    if (p.vec != 2) {          // rows out of line: through LDS, one output per lane
      constexpr int NT = 2 * WF;
      static_assert(W * flush_floats(NT) * 4 <= Sh::LDS);
      float* buf = (float*)lds + wave * flush_floats(NT);
#pragma unroll
      for (int i = 0; i < AF; ++i)
#pragma unroll
        for (int q = 0; q < 2; ++q)
          flush_half<NT, WF>(p, buf, acc[i], q, p.M - mw - 32 * i - 16 * q, nw,
                             [&](int lr) SWQ_INLINE { return (int64_t)(mw + 32 * i + 16 * q + lr); });
      meet();
    }
    block += gridDim.x;
    const bool more = aim(block);
    if (more) begin();
    if (p.vec == 2) {
      if (p.out_type == kTypeF32) store_wide<kTypeF32, AF, WF>(p, acc, mw, nw);
      else if (p.out_type == kTypeF16) store_wide<kTypeF16, AF, WF>(p, acc, mw, nw);
      else store_wide<kTypeBf16, AF, WF>(p, acc, mw, nw);
    }
    if (!more) break;
  }
}

// Few outputs: 16 x 16 per block, everything straight to registers; the W
// waves take steps of 128 inputs in turn, U of them in flight, and add their
// sums in wave order.  (16 x 16 x 128 MFMA: lane 16 h + r holds row r's block h.)
// 200 x 2080 x 1001: 6.6 us; 33 x 1024 x 1001 3.3, two loads' latency and the launch.
template <int W, int U>
__global__ __launch_bounds__(64 * W) void mx4_matmul_few_kernel(Mx4Matmul p) {
  __shared__ f32x4 lds[W * 64];
#ifdef SWQ_LDS_POISON
  lds_poison(lds, sizeof(lds), kPoisonFloat);
  __syncthreads();
#endif
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, h = lane >> 4;
  const int ntn = (p.N + 15) / 16;
  const int m0 = (blockIdx.x / ntn) * 16, n0 = (blockIdx.x % ntn) * 16;
  const int rows = min(16, p.M - m0), cols = min(16, p.N - n0);
  const int blocks = p.K / 32, steps = (blocks + 3) / 4;
  // rows past the end read zeros and touch no memory
  const __amdgpu_buffer_rsrc_t ra = buffer(p.a + (int64_t)m0 * (p.K / 8), rows * (p.K / 2));
  const __amdgpu_buffer_rsrc_t rw = buffer(p.w + (int64_t)n0 * (p.K / 8), cols * (p.K / 2));
  const __amdgpu_buffer_rsrc_t sra = buffer(p.sa + (int64_t)m0 * blocks, rows * blocks);
  const __amdgpu_buffer_rsrc_t srw = buffer(p.s + (int64_t)n0 * blocks, cols * blocks);
  const uint32_t off = r * (p.K / 2) + h * 16;
  const uint32_t soff = r * blocks + h;
  f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int t0 = wave; t0 < steps; t0 += W * U) {
    u32x4 a[U], w[U];
    uint32_t fa[U], fw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = t0 + u * W;
      const bool in = 4 * t + h < blocks;
      a[u] = load16(ra, in ? off + t * 64 : kNowhere);
      w[u] = load16(rw, in ? off + t * 64 : kNowhere);
      fa[u] = load1(sra, in ? soff + 4 * t : kNowhere);
      fw[u] = load1(srw, in ? soff + 4 * t : kNowhere);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) acc = mfma_mx4(w[u], fw[u], a[u], fa[u], acc);
  }
  lds[wave * 64 + lane] = acc;
  __syncthreads();
  if (wave != 0 || r >= rows || n0 + 4 * h >= p.N) return;
  f32x4 y = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int v = 0; v < W; ++v) y += lds[v * 64 + lane];
  store4(p.out, (int64_t)(m0 + r) * p.N, n0 + 4 * h, p.N, p.vec, y, p.out_type);
}

}  // namespace

static int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// What a product runs on: the few-row kernel up to 24 rows, 32 of binary16 x (a grouped product: 10 of an average
// expert, 20 of binary16 x; 32 experts, K x N = 2048 x 1408, 8 / 16 / 32 rows each:
// few-row kernel 22 / 28 / 45 us, tiles 28 / 35 / 29), else the tile shape whose fullest
// CU is done first.  Measured on one MI355X, a CU takes 1.77 us per chunk of a 128 x 256 tile, 0.98 of a 128 x 128 and
// 0.62 of a 64 x 128 one, however many blocks it holds (bf16 x; us):
//   rows x K x N          64 x 128   128 x 128   128 x 256
//   1024 x 5632 x 2048        34         48          82
//   512 x 2048 x 5632         24         21          36
//   6144 x 2048 x 1408        54         49          56
//   2048 x 4096 x 14336      286        217         218
//   8192 x 2560 x 10240      471        391         353
// binary16 x, whose rows are two operands, takes 64 rows a tile: 0.95 us per chunk of 64 x 128 and 1.66 of
// 64 x 256, 2.2 where a CU has a single one (us; one to two rounds of tiles, three and more):
//   rows x K x N          64 x 128   64 x 256      rows x K x N          64 x 128   64 x 256
//   256 x 4096 x 14336       64         70         512 x 4096 x 14336      121        111
//   384 x 2048 x 5632        37         40         1024 x 2048 x 5632       57         64
//   768 x 4096 x 4096        68         73         2048 x 2560 x 10240     189        168
// and its few-row kernel holds up to 32 rows (32 x K x N = 4096 x 4096, 4096 x 14336, 2560 x 10240, 5632 x 2048: 15 / 23 /
// 18 / 18 us against 18 / 28 / 20 / 17 by tiles, bf16 13 / 20 / 18 / 16 against 14 / 20 / 15 / 14).
// Where their tiles leave CUs idle the 64 x 128 kernel splits K (K x N = 5632 x 2048,
// 32 / 64 / 256 rows: few-row kernel 15 / 26 / 27, split 13 / 15 / 19; 8192 x 512 20 / 35 / 35 against
// 14 / 15 / 18).  On small weights, K N <= 2^20, the second launch costs more than
// it gives: 1024 x 1024, 256 rows, few-row 8, split 11.
int mx4_gemm_kind(const MxGemm& p) {
  const int64_t each = p.rows / p.E;
  const bool f16 = p.xsrc != kXBf16;
  if (each <= (p.E == 1 ? (f16 ? 32 : 24) : f16 ? 20 : 10)) return kFew;
  if (p.E == 1 && each <= 256 && (int64_t)p.K * p.N <= (1 << 20)) return kFew;
  const int64_t part = p.E == 1 ? 0 : p.E / 2;           // half a tile per expert for its last, partial one
  const int64_t n = p.w2 ? 2 * (int64_t)p.N : p.N, cus = device_cus();
  const auto rounds = [&](int bm, int bn) { return ceil_div((ceil_div(p.rows, bm) + part) * ceil_div(n, bn), cus); };
  if (f16) {
    const int64_t large = rounds(64, 256);
    return 95 * rounds(64, 128) <= (large == 1 ? 220 : 166 * large) ? kSmallTiles : kLargeTiles;
  }
  const int64_t large = 177 * rounds(128, 256), mid = 98 * rounds(128, 128), small = 62 * rounds(64, 128);
  if (small <= mid && small <= large) return kSmallTiles;
  return mid < large ? kMidTiles : kLargeTiles;
}

// K split of 64 x 128 tiles that leave half the CUs without one: at least four chunks each, at most 16 ways.
int mx4_gemm_splits(const MxGemm& p) {
  if (p.kind != kSmallTiles || p.tiles || p.offsets || p.w2) return 1;
  const int64_t tiles = ceil_div(p.rows, 64) * ceil_div(p.N, 128), chunks = ceil_div(p.K, 128);
  int64_t n = std::min<int64_t>(std::min<int64_t>(device_cus() / tiles, chunks / 4), 16);
  if (n < 2) return 1;
  return (int)ceil_div(chunks, ceil_div(chunks, n));     // no empty split
}

// Row tiles of 16 of the few-row kernel, by the rows of an average expert.
static int few_tiles(const MxGemm& p) {
  const int64_t each = p.rows / p.E;
  return p.E == 1 ? (p.rows <= 16 ? 1 : p.rows <= 32 ? 2 : 4) : each <= 8 ? 1 : each <= 20 ? 2 : 4;
}

int mx4_gemm_tile(const MxGemm& p) {
  const int k = p.kind;
  return k == kFew ? 16 * few_tiles(p) : k == kSmallTiles || p.xsrc != kXBf16 ? 64 : 128;
}

bool mx4_gemm_takes_planes(const MxGemm& p) { return p.kind != kFew; }

// A launch of 2^32 threads or more is cut off without an error.
static bool one_launch(int64_t blocks, int threads) { return blocks * threads < (int64_t(1) << 32); }

template <int MF, int NF, int WM, int WN, int NP, int S, bool FUSED>
static hipError_t launch_tiled(const MxGemm& p, hipStream_t st) {
  constexpr int BM = 16 * MF * WM, BNO = 16 * NF * WN / (FUSED ? 2 : 1);
  const int64_t ntm = p.max_tiles ? p.max_tiles : ceil_div(p.rows, BM), ntn = ceil_div(p.N, BNO);
  const int64_t blocks = ceil_div(ntm * ntn, 8) * 8;
  if (!one_launch(blocks, 64 * WM * WN)) return hipErrorInvalidConfiguration;
  if (p.check_only) return hipSuccess;
  if constexpr (!FUSED && MF == 4 && NF == 2) {
    if (p.splits > 1) {
      // K split: float32 partial sums [split][row][column] in the workspace, added in split order
      MxGemm q = p;
      q.split_chunks = ((p.K + 127) / 128 + p.splits - 1) / p.splits;
      q.out = p.parts;
      q.out_type = kTypeF32;
      q.res = nullptr;
      q.vec = p.N % 8 == 0 ? 2 : 0;
      mx4_gemm_kernel<MF, NF, WM, WN, NP, S, FUSED, true>
          <<<dim3((unsigned)blocks, (unsigned)p.splits), 64 * WM * WN, 0, st>>>(q);
      const int64_t threads = (int64_t)p.rows * ((p.N + 3) / 4);
      mx4_join_kernel<<<dim3((unsigned)((threads + 255) / 256)), 256, 0, st>>>(p);
      return hipGetLastError();
    }
  }
  mx4_gemm_kernel<MF, NF, WM, WN, NP, S, FUSED, false><<<dim3((unsigned)blocks), 64 * WM * WN, 0, st>>>(p);
  return hipGetLastError();
}

template <int RT, int CT, int XS, bool FUSED, int W, int U>
static hipError_t launch_few_as(const MxGemm& p, hipStream_t st) {
  const int64_t ntn = (p.N + 16 * CT - 1) / (16 * CT);
  const int64_t ntm = p.max_tiles ? p.max_tiles : ceil_div(p.rows, 16 * RT);
  if (!one_launch(ntm * ntn, 64 * W)) return hipErrorInvalidConfiguration;
  if (p.check_only) return hipSuccess;
  mx4_few_kernel<RT, CT, XS, FUSED, W, U><<<dim3((unsigned)(ntm * ntn)), 64 * W, 0, st>>>(p);
  return hipGetLastError();
}

// Column tiles per block: as many as leave seven eighths of the CUs a block (more columns
// read x less often).
template <int RT, int XS, bool FUSED>
static hipError_t launch_few_rt(const MxGemm& p, hipStream_t st) {
  constexpr int D = FUSED ? 2 : 1;
  const int64_t tiles = p.max_tiles ? std::min<int64_t>(p.max_tiles, p.rows) : ceil_div(p.rows, 16 * RT);
  const int64_t need = device_cus() * 7 / 8;
  if (p.N / (16 * 4 / D) * tiles >= need) return launch_few_as<RT, 4 / D, XS, FUSED, 8, 1>(p, st);
  if (p.N / (16 * 2 / D) * tiles >= need || FUSED)
    return launch_few_as<RT, 2 / D, XS, FUSED, 8, RT == 1 ? 2 : 1>(p, st);
  if constexpr (!FUSED) return launch_few_as<RT, 1, XS, FUSED, 8, RT <= 2 ? 2 : 1>(p, st);
  return hipErrorInvalidValue;
}

template <int XS, bool FUSED, int W>
static hipError_t launch_row(const MxGemm& p, hipStream_t st) {
  const int64_t blocks = (int64_t)p.rows * ((p.N + 15) / 16);
  if (!one_launch(blocks, 64 * W)) return hipErrorInvalidConfiguration;
  if (p.check_only) return hipSuccess;
  mx4_row_kernel<XS, FUSED, W><<<dim3((unsigned)blocks), 64 * W, 0, st>>>(p);
  return hipGetLastError();
}

template <int XS, bool FUSED>
static hipError_t launch_few(const MxGemm& p, hipStream_t st) {
  if constexpr (XS != kXPlanes)                    // (planes: the hidden tensor of experts by tiles, else mx4_down_kernel)
    if (!p.max_tiles && (p.ids || p.rows == 1))    // rows one by one; four waves cover 2048 inputs at once
      return p.K <= 4 * kRowU * 128 ? launch_row<XS, FUSED, 4>(p, st) : launch_row<XS, FUSED, 8>(p, st);
  const int rt = few_tiles(p);
  return rt == 1 ? launch_few_rt<1, XS, FUSED>(p, st) : rt == 2 ? launch_few_rt<2, XS, FUSED>(p, st)
                                                                : launch_few_rt<4, XS, FUSED>(p, st);
}

template <bool FUSED>
static hipError_t launch_gemm(const MxGemm& p, hipStream_t st) {
  const int k = p.kind;
  if (k == kFew) {
    if constexpr (!FUSED)
      if (p.xsrc == kXPlanes) return launch_few<kXPlanes, false>(p, st);
    return p.xsrc == kXBf16 ? launch_few<kXBf16, FUSED>(p, st) : launch_few<kXF16, FUSED>(p, st);
  }
  if (p.xsrc != kXBf16)
    return k == kSmallTiles ? launch_tiled<4, 2, 1, 4, 2, 2, FUSED>(p, st)
                            : launch_tiled<4, 4, 1, 4, 2, 2, FUSED>(p, st);
  return k == kSmallTiles ? launch_tiled<4, 2, 1, 4, 1, 4, FUSED>(p, st)
         : k == kMidTiles ? launch_tiled<8, 2, 1, 4, 1, 2, FUSED>(p, st)
                          : launch_tiled<8, 4, 1, 4, 1, 2, FUSED>(p, st);
}

hipError_t launch_mx4_gemm(const MxGemm& p, hipStream_t st) {
  return p.w2 ? launch_gemm<true>(p, st) : launch_gemm<false>(p, st);
}

hipError_t launch_mx4_down(const MxGemm& p, const float* weights, int k, hipStream_t st) {
  constexpr int W = 16;
  const int64_t blocks = (int64_t)(p.rows / k) * ((p.N + 15) / 16);
  if (!one_launch(blocks, 64 * W)) return hipErrorInvalidConfiguration;
  if (p.check_only) return hipSuccess;
  // as many waves per slot as leave no slot waiting, and no more than it has chunks for
  int share = W;
  while (share > 1 && (share * k > W || (share - 1) * kRowU * 128 >= p.K)) share >>= 1;
  const dim3 grid((unsigned)blocks);
  if (p.xsrc == kXPlanes) mx4_down_kernel<kXPlanes, W><<<grid, 64 * W, 0, st>>>(p, weights, k, share);
  else mx4_down_kernel<kXBf16, W><<<grid, 64 * W, 0, st>>>(p, weights, k, share);
  return hipGetLastError();
}

namespace {
// Binary16 x as two planes of bf16, once, for products whose tiles read a row of x many times (six bytes
// of traffic per input; few rows are split where they are read).
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
  constexpr int64_t kLaunch = int64_t(1) << 30;          // a launch holds fewer than 2^32 threads
  for (int64_t i = 0; i < n / 8; i += kLaunch) {
    const int64_t n8 = std::min(kLaunch, n / 8 - i);
    mx4_split_kernel<<<dim3((unsigned)((n8 + 255) / 256)), 256, 0, st>>>(
        (const f16x8*)x + i, n8, (bf16x8*)planes + i, (bf16x8*)(planes + plane) + i);
  }
  return hipGetLastError();
}

static int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

struct MatmulConfig {
  int bm, bn;
  hipError_t (*launch)(const Mx4Matmul&, const uint16_t*, int, int, hipStream_t);
};

template <int AF, int WF, int WM, int WN, int S, int OCC>
static hipError_t launch_matmul_as(const Mx4Matmul& p, const uint16_t* ws, int stages, int pad_a, hipStream_t st) {
  using Sh = MmShape<AF, WF, WM, WN, S>;
  const int64_t tiles = (int64_t)((p.M + Sh::BM - 1) / Sh::BM) * ((p.N + Sh::BN - 1) / Sh::BN);
  if (tiles >= (1LL << 30)) return hipErrorInvalidValue;
  const int64_t blocks = std::min<int64_t>(round_up(tiles, 8), (int64_t)device_cus() / 8 * 8 * OCC);
  mx4_matmul_kernel<AF, WF, WM, WN, S, OCC>
      <<<dim3((unsigned)blocks), 64 * WM * WN, 0, st>>>(p, ws, stages, pad_a);
  return hipGetLastError();
}

// Tile shapes.  Measured (us; 8192 x 2560 x 10240, 2048 x 4096 x 14336, 200 x 2080 x 1001
// with its scale layout):
//   256 x 256   149   77   27     eight waves; the others four, and two blocks a CU
//   128 x 128   197   90   16
//    64 x  64   299  140    8.9   seven stages deep
// (the larger tile reads fewer bytes from L2; 128 x 256 took 179, 87 and 23).  256 x 256 where it gives three fifths of the CUs a tile, 128 x 128
// where it gives half of them one, else 64 x 64.
static const MatmulConfig kMatmul[] = {
    {256, 256, launch_matmul_as<4, 2, 2, 4, 4, 1>},
    {128, 128, launch_matmul_as<2, 2, 2, 2, 4, 2>},
    {64, 64, launch_matmul_as<1, 1, 2, 2, 7, 2>},
};

// The tiles address their operands with 32-bit byte offsets.  An operand past them is taken in slabs of
// rows, about equal ones of whole tiles, each with launches of its own: 1114112 x 8192 x 512
// (4.25 GiB of codes) in two slabs 3.2 ms (2.9 PFLOP/s);
// the kernel for few outputs, which needs no slabs, takes 60.
constexpr int64_t kSlabBytes = (int64_t(1) << 32) - 16;
static int64_t slab_rows(int64_t rows, int64_t K) {
  const int64_t slabs = ceil_div(rows, kSlabBytes / (K / 2) / 256 * 256);
  return slabs < 2 ? rows : round_up(ceil_div(rows, slabs), 256);
}
static Mx4Matmul slab(const Mx4Matmul& p, int64_t m, int64_t n) {      // the one that starts at row m, column n
  Mx4Matmul q = p;
  q.a += m * (p.K / 8);
  q.sa += m * (p.K / 32);
  q.w += n * (p.K / 8);
  q.s += n * (p.K / 32);
  q.out = (char*)p.out + (m * p.ld + n) * type_bytes(p.out_type);
  q.M = (int)std::min(slab_rows(p.M, p.K), p.M - m);
  q.N = (int)std::min(slab_rows(p.N, p.K), p.N - n);
  return q;
}

static const MatmulConfig* matmul_config(const Mx4Matmul& p) {
  const int64_t cus = device_cus();
  // Up to two 16 x 16 tiles a CU, or four with little K: no scale layout, no LDS, one launch.
  // Against the 64 x 64 tiles with their scale layout (us; tiles, M x K x N):
  //   256  33 x 4096 x 1001    5.7 against 10.5      1024  64 x 1024 x 4096    6.3 against  6.5
  //   512  24 x 8192 x 4096   14.8 against 15.5       819  200 x 2080 x 1001   5.9 against  8.9
  //   896  16 x 4096 x 14336  16.2 against 14.1      1024  32 x 4096 x 8192   16.1 against 11.4
  const int64_t small = ceil_div(p.M, 16) * ceil_div(p.N, 16);
  if (small <= 2 * cus || (small <= 4 * cus && (int64_t)p.M * p.N * p.K <= (int64_t(1) << 29))) return nullptr;
  const Mx4Matmul q = slab(p, 0, 0);
  const auto tiles = [&](const MatmulConfig& c) { return ceil_div(q.M, c.bm) * ceil_div(q.N, c.bn); };
  return 5 * tiles(kMatmul[0]) >= 3 * cus   ? &kMatmul[0]
         : 2 * tiles(kMatmul[1]) >= cus ? &kMatmul[1]
                                          : &kMatmul[2];
}

int64_t mx4_matmul_workspace(const Mx4Matmul& p) {
  const MatmulConfig* c = matmul_config(p);
  const Mx4Matmul q = slab(p, 0, 0);         // the largest; the others' scales take its place in turn
  return c ? (round_up(q.M, c->bm) + round_up(q.N, c->bn)) * ((p.K + 127) / 128) * 4 : 0;
}

hipError_t launch_mx4_matmul(const Mx4Matmul& p, void* ws, hipStream_t st) {
  const MatmulConfig* c = matmul_config(p);
  if (!c) {                                  // few blocks, by the rule above
    const int64_t tiles = ceil_div(p.N, 16) * ceil_div(p.M, 16);
    mx4_matmul_few_kernel<8, 2><<<dim3((unsigned)tiles), 512, 0, st>>>(p);
    return hipGetLastError();
  }
  const int stages = (p.K + 127) / 128;
  const int64_t ms = slab_rows(p.M, p.K), ns = slab_rows(p.N, p.K);
  for (int64_t m = 0; m < p.M; m += ms)
    for (int64_t n = 0; n < p.N; n += ns) {
      const Mx4Matmul q = slab(p, m, n);
      const int pad_a = (int)round_up(q.M, c->bm), pad_w = (int)round_up(q.N, c->bn);
      const int64_t threads = (int64_t)(pad_a + pad_w) * stages;
      mx4_scale_kernel<<<dim3((unsigned)((threads + 255) / 256)), 256, 0, st>>>(
          q.sa, q.M, q.s, q.N, q.K / 32, stages, pad_a, pad_w, (uint16_t*)ws);
      const hipError_t rc = c->launch(q, (const uint16_t*)ws, stages, pad_a, st);
      if (rc != hipSuccess) return rc;
    }
  return hipSuccess;
}

}  // namespace swq
