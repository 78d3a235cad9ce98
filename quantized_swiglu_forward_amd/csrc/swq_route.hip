// The router's choice, the order of a product grouped by expert, and the sum
// over a token's experts.
#include <algorithm>

#include "swq_mx4.h"
#include "swq_mx4_device.h"

namespace swq {
namespace {

// Routing weights (values fixed by the public header).
enum : int { kRouteSoftmax = 0, kRouteSoftmaxChosen = 1, kRouteSigmoid = 2, kRouteSigmoidChosen = 3 };

constexpr int kMaxExperts = 1024;

// A chosen logit's weight before the division by the sum: e^(v - top), or the sigmoid
// e^min(v, 0) / (1 + e^-|v|), over the chosen ones times e^-min(top, 0), so that
// very low logits do not make it 0 / 0.
__device__ __forceinline__ float routing_term(float v, float top, int scoring) {
  if (scoring <= kRouteSoftmaxChosen) return expf(v - top);
  const float from = scoring == kRouteSigmoidChosen ? fminf(top, 0.0f) : 0.0f;
  return expf(fminf(v, 0.0f) - from) / (1.0f + expf(-fabsf(v)));
}

constexpr float kMaxFloat = 3.402823466e38f;

// A logit as an unsigned number that orders like it: 0 for -inf and NaN (never
// chosen), equal for both zeros, +inf above everything.
template <int TYPE>
struct LogitKey {             // float32: the value's 32 bits
  static __device__ __forceinline__ uint32_t of(uint32_t bits) {
    if (bits == 0x80000000u) bits = 0;
    if (bits == 0x7F800000u) bits = 0x7F7FFFFFu;       // +inf counts as the largest float32
    const bool out = (bits & 0x7FFFFFFFu) > 0x7F800000u || bits == 0xFF800000u;
    return out ? 0u : bits ^ ((bits >> 31) ? 0xFFFFFFFFu : 0x80000000u);
  }
  static __device__ __forceinline__ float value(uint32_t key) {
    return __uint_as_float(key ^ ((key >> 31) ? 0x80000000u : 0xFFFFFFFFu));
  }
};
template <int TYPE>
struct LogitKey16 {           // bf16, binary16: the 16 bits
  static constexpr uint32_t kInf = TYPE == kTypeF16 ? 0x7C00u : 0x7F80u;
  static __device__ __forceinline__ uint32_t of(uint32_t bits) {
    if (bits == 0x8000u) bits = 0;
    const bool out = (bits & 0x7FFFu) > kInf || bits == (kInf | 0x8000u);
    return out ? 0u : (bits ^ ((bits >> 15) ? 0xFFFFu : 0x8000u));
  }
  static __device__ __forceinline__ float value(uint32_t key) {
    return fminf(from_16((uint16_t)(key ^ ((key >> 15) ? 0x8000u : 0xFFFFu)), TYPE), kMaxFloat);
  }
};

// op over a group of G lanes (16 neighbours, or the wave); every lane gets the result.
template <int ROT>
__device__ __forceinline__ uint32_t rotate16(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + ROT, 0xF, 0xF, true);
}
template <int G, class Op>
__device__ __forceinline__ uint32_t over_group(uint32_t v, Op op) {
  v = op(v, rotate16<8>(v));
  v = op(v, rotate16<4>(v));
  v = op(v, rotate16<2>(v));
  v = op(v, rotate16<1>(v));
  if constexpr (G == 64) {
    v = op(v, (uint32_t)__shfl_xor((int)v, 16));
    v = op(v, (uint32_t)__shfl_xor((int)v, 32));
  }
  return v;
}
__device__ __forceinline__ uint32_t max_u32(uint32_t a, uint32_t b) { return max(a, b); }
__device__ __forceinline__ uint32_t min_u32(uint32_t a, uint32_t b) { return min(a, b); }
__device__ __forceinline__ uint32_t add_f32(uint32_t a, uint32_t b) {
  return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
}

// G lanes per token, R logits per lane, k rounds of a maximum over the group.  A
// 16-bit logit and its index make one 32-bit key that orders by value, then by
// the lower index; float32 takes a second reduction, over the indices of the
// largest.  VEC: a lane's logits are neighbours, loaded 16 bytes at a time; else lane l has
// l, l + G, ...  KR: chosen experts per lane (k <= 16 KR).
//
// Bound by the k rounds' chain of row rotations, not by bytes: 8192 tokens of 256 logits, top 8, 7.0 us (4.7 MB);
// one token of 64 2.5 us, the launch and one load.  Sixteen lanes a token give 2048 waves where a wave a
// token gives 8192 and longer reductions: 22 us.
template <int TYPE, int G, int R, int KR, bool VEC>
__global__ __launch_bounds__(256) void route_kernel(const void* __restrict__ logits, int64_t T, int E, int k,
                                                    int scoring, int* __restrict__ ids, float* __restrict__ weights) {
  constexpr bool F32 = TYPE == kTypeF32;
  const int lane = threadIdx.x & (G - 1), l16 = threadIdx.x & 15;
  const int64_t t = ((int64_t)blockIdx.x * 256 + threadIdx.x) / G;
  const bool live = t < T;
  const int64_t row = (live ? t : T - 1) * E;
  // (no lane leaves early: the reductions take every lane of their group)
  const auto index = [&](int i) { return VEC ? lane * R + i : i * G + lane; };
  uint32_t key[R];
  if constexpr (VEC) {
    if constexpr (F32) {
#pragma unroll
      for (int i = 0; i < R; i += 4) {
        u32x4 q = {0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u};
        if (lane * R + i < E) q = *(const u32x4*)((const uint32_t*)logits + row + lane * R + i);
#pragma unroll
        for (int j = 0; j < 4; ++j) key[i + j] = LogitKey<TYPE>::of(q[j]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < R; i += 8) {
        u32x4 q = {0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu};
        if (lane * R + i < E) q = *(const u32x4*)((const uint16_t*)logits + row + lane * R + i);
#pragma unroll
        for (int j = 0; j < 8; ++j) key[i + j] = LogitKey16<TYPE>::of((q[j >> 1] >> (16 * (j & 1))) & 0xFFFFu);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const bool in = index(i) < E;
      if constexpr (F32) key[i] = LogitKey<TYPE>::of(in ? ((const uint32_t*)logits)[row + index(i)] : 0xFF800000u);
      else key[i] = LogitKey16<TYPE>::of(in ? ((const uint16_t*)logits)[row + index(i)] : 0xFFFFu);
    }
  }
  const auto value = [&](uint32_t v) {
    if constexpr (F32) return LogitKey<TYPE>::value(v);
    else return LogitKey16<TYPE>::value(v);
  };

  float top = 0.0f, sum = 0.0f;
  if (scoring == kRouteSoftmax) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < R; ++i) m = max(m, key[i]);
    m = over_group<G>(m, max_u32);
    top = value(m);
    // (small terms need no more than the hardware's exp2 gives: their error is below the sum's own rounding)
#pragma unroll
    for (int i = 0; i < R; ++i)
      sum += key[i] ? __builtin_amdgcn_exp2f((value(key[i]) - top) * 1.4426950408889634f) : 0.0f;
    sum = __uint_as_float(over_group<G>(__float_as_uint(sum), add_f32));
  }
  if constexpr (!F32) {
#pragma unroll
    for (int i = 0; i < R; ++i) key[i] = key[i] ? key[i] << 16 | (0xFFFFu - (uint32_t)index(i)) : 0u;
  }

  int id[KR];
  float w[KR], chosen = 0.0f;
#pragma unroll
  for (int s = 0; s < KR; ++s) {
    id[s] = -1;
    w[s] = 0.0f;
    for (int j = 16 * s; j < 16 * s + 16 && j < k; ++j) {
      uint32_t best = 0;
#pragma unroll
      for (int i = 0; i < R; ++i) best = max(best, key[i]);
      best = over_group<G>(best, max_u32);
      uint32_t at;
      float v;
      if constexpr (F32) {
        at = 0xFFFFu;
#pragma unroll
        for (int i = R - 1; i >= 0; --i) at = key[i] == best ? (uint32_t)index(i) : at;
        at = over_group<G>(at, min_u32);
        v = value(best);
#pragma unroll
        for (int i = 0; i < R; ++i) key[i] = (uint32_t)index(i) == at ? 0u : key[i];
      } else {
        at = 0xFFFFu - (best & 0xFFFFu);
        v = value(best >> 16);
#pragma unroll
        for (int i = 0; i < R; ++i) key[i] = key[i] == best ? 0u : key[i];
      }
      if (best != 0) {                         // else only -inf is left
        if (j == 0) top = v;
        const float term = routing_term(v, top, scoring);
        chosen += term;
        if (l16 == (j & 15)) id[s] = (int)at, w[s] = term;
      }
    }
  }
  if (!live || lane >= 16) return;
  const float by = scoring == kRouteSoftmax ? sum : scoring == kRouteSigmoid ? 1.0f : chosen;
#pragma unroll
  for (int s = 0; s < KR; ++s) {
    const int j = 16 * s + l16;
    if (j < k) {
      ids[t * k + j] = id[s];
      weights[t * k + j] = id[s] < 0 ? 0.0f : w[s] / by;
    }
  }
}

// Order of the rows of a grouped product and its tiles.  With
// ids: the slots of each expert's rows (their order within an expert decides
// no result: every output row depends on its own input row alone).  With
// offsets: the groups as given, made non-decreasing and cut at P; the rows
// before the first and after the last group become tiles of no expert.
// Thread t holds expert t.  The order's scattered stores, one line each, bound it
// (32768 rows of 64 experts in one block: 21 us), so from kPlanSplit rows on each of
// kPlanBlocks blocks counts all ids and stores for the experts e = its number modulo the
// blocks: 12 us there; 4096 rows 6.1 -> 5.9, 2048 5.2 -> 5.7.
constexpr int kPlanThreads = 1024, kPlanAhead = 8, kPlanBlocks = 8, kPlanSplit = 4096;

// Inclusive sum (or maximum) over the threads of a block.
template <bool MAX>
__device__ __forceinline__ int block_scan(int v, int* wave_total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(v, d);
    if (lane >= d) v = MAX ? max(v, o) : v + o;
  }
  if (lane == 63) wave_total[wave] = v;
  __syncthreads();
  int before = MAX ? INT32_MIN : 0;
  for (int w = 0; w < wave; ++w) before = MAX ? max(before, wave_total[w]) : before + wave_total[w];
  __syncthreads();
  return MAX ? max(v, before) : v + before;
}

__global__ __launch_bounds__(kPlanThreads) void plan_kernel(RoutePlan p) {
  __shared__ int count[kMaxExperts], next[kMaxExperts], total[kPlanThreads / 64];
#ifdef SWQ_LDS_POISON
  lds_poison(count, sizeof(count), kPoisonExp);
  lds_poison(next, sizeof(next), kPoisonExp);
  lds_poison(total, sizeof(total), kPoisonExp);
  __syncthreads();
#endif
  const int t = threadIdx.x, mask = gridDim.x - 1;
  int rows = 0, first = 0, last = 0;           // of expert t; the end of the last expert's rows
  if (p.ids) {
    if (t < p.E) count[t] = 0;
    __syncthreads();
    for (int i0 = t; i0 < p.P; i0 += kPlanThreads * kPlanAhead) {
      int e[kPlanAhead];
#pragma unroll
      for (int j = 0; j < kPlanAhead; ++j) e[j] = i0 + j * kPlanThreads < p.P ? p.ids[i0 + j * kPlanThreads] : -1;
#pragma unroll
      for (int j = 0; j < kPlanAhead; ++j)
        if (e[j] >= 0 && e[j] < p.E) atomicAdd(&count[e[j]], 1);
    }
    __syncthreads();
    rows = t < p.E ? count[t] : 0;
  } else {
    const int start = block_scan<true>(t < p.E ? min(max(p.offsets[t], 0), p.P) : 0, total);
    if (t < p.E) next[t] = start;
    if (t == p.E - 1) count[0] = max(start, min(max(p.offsets[p.E], 0), p.P));
    __syncthreads();
    last = count[0];
    first = start;
    rows = t < p.E ? (t + 1 < p.E ? next[t + 1] : last) - start : 0;
  }
  const int tiles = (rows + p.tile - 1) / p.tile;
  if (p.ids) first = block_scan<false>(rows, total) - rows;
  const int tile_end = block_scan<false>(tiles, total);
  for (int i = 0; (t & mask) == blockIdx.x && i < tiles; ++i)
    p.tiles[tile_end - tiles + i] = RowTile{t, first + i * p.tile, min(p.tile, rows - i * p.tile), 0};
  if (p.ids) {
    if (blockIdx.x == 0 && t == kPlanThreads - 1) *p.ntiles = tile_end;
    if (t < p.E) next[t] = first;
    __syncthreads();
    for (int i0 = t; i0 < p.P; i0 += kPlanThreads * kPlanAhead) {
      int e[kPlanAhead];
#pragma unroll
      for (int j = 0; j < kPlanAhead; ++j) e[j] = i0 + j * kPlanThreads < p.P ? p.ids[i0 + j * kPlanThreads] : -1;
#pragma unroll
      for (int j = 0; j < kPlanAhead; ++j)
        if (e[j] >= 0 && e[j] < p.E && (e[j] & mask) == blockIdx.x)
          p.perm[atomicAdd(&next[e[j]], 1)] = i0 + j * kPlanThreads;
    }
  } else if (t == kPlanThreads - 1) {          // rows of no expert, before and after the groups
    int n = tile_end;
    for (int i = 0; i < next[0]; i += p.tile) p.tiles[n++] = RowTile{-1, i, min(p.tile, next[0] - i), 0};
    for (int i = last; i < p.P; i += p.tile) p.tiles[n++] = RowTile{-1, i, min(p.tile, p.P - i), 0};
    *p.ntiles = n;
  }
}

// One thread per V neighbours of an output row: the k partial rows are read four slots
// at a time, each slot's id and weight first, and added in the slots' order in float32 before the one
// rounding.  Bound by the partial rows: 4096 tokens of 8, 1024 columns, 134 MB: 26 us, 5.3 TB/s from the
// last-level cache.
template <int V>
__global__ __launch_bounds__(256) void combine_kernel(const float* __restrict__ part, const int* __restrict__ ids,
                                                      const float* __restrict__ weights,
                                                      const uint16_t* __restrict__ res, int64_t T, int k, int E, int N,
                                                      int64_t ld, int type, int out_type, void* __restrict__ out) {
  const int per = N / V;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t t = i / per;
  const int n = (int)(i - t * per) * V;
  if (t >= T) return;
  const int64_t at = t * ld + n;
  float y[V];
#pragma unroll
  for (int v = 0; v < V; ++v) y[v] = res ? from_16(res[at + v], type) : 0.0f;
  for (int j0 = 0; j0 < k; j0 += 4) {
    float p[4][V], w[4];
    bool on[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t slot = t * k + j0 + j;
      const int e = j0 + j < k ? ids[slot] : -1;
      on[j] = e >= 0 && e < E;
      w[j] = on[j] ? weights[slot] : 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) p[j][v] = 0.0f;
      if (on[j]) {
        if constexpr (V == 4) {
          const f32x4 q = *(const f32x4*)(part + slot * N + n);
#pragma unroll
          for (int v = 0; v < V; ++v) p[j][v] = q[v];
        } else {
          p[j][0] = part[slot * N + n];
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int v = 0; v < V; ++v) y[v] = on[j] ? fmaf(w[j], p[j][v], y[v]) : y[v];
  }
  if constexpr (V == 4) {
    store4(out, at - n, n, N, true, (f32x4){y[0], y[1], y[2], y[3]}, out_type);
  } else if (out_type == kTypeF32) {
    ((float*)out)[at] = y[0];
  } else {
    ((uint16_t*)out)[at] = to_16(y[0], out_type);
  }
}

}  // namespace

template <int TYPE, int G, int R, int KR>
static hipError_t launch_route_as(const void* logits, int64_t T, int E, int k, int scoring, int* ids, float* weights,
                                  hipStream_t st) {
  constexpr int WIDE = TYPE == kTypeF32 ? 4 : 8;
  const dim3 grid((unsigned)((T * G + 255) / 256));
  if constexpr (R % WIDE == 0) {
    if (E % WIDE == 0 && (uintptr_t)logits % 16 == 0) {
      route_kernel<TYPE, G, R, KR, true><<<grid, 256, 0, st>>>(logits, T, E, k, scoring, ids, weights);
      return hipGetLastError();
    }
  }
  route_kernel<TYPE, G, R, KR, false><<<grid, 256, 0, st>>>(logits, T, E, k, scoring, ids, weights);
  return hipGetLastError();
}

template <int TYPE, int KR>
static hipError_t launch_route_type(const void* logits, int64_t T, int E, int k, int scoring, int* ids, float* weights,
                                    hipStream_t st) {
  if (E <= 64) return launch_route_as<TYPE, 16, 4, KR>(logits, T, E, k, scoring, ids, weights, st);
  if (E <= 128) return launch_route_as<TYPE, 16, 8, KR>(logits, T, E, k, scoring, ids, weights, st);
  if (E <= 256) return launch_route_as<TYPE, 16, 16, KR>(logits, T, E, k, scoring, ids, weights, st);
  if (E <= 512) return launch_route_as<TYPE, 64, 8, KR>(logits, T, E, k, scoring, ids, weights, st);
  return launch_route_as<TYPE, 64, 16, KR>(logits, T, E, k, scoring, ids, weights, st);
}

template <int TYPE>
static hipError_t launch_route_k(const void* logits, int64_t T, int E, int k, int scoring, int* ids, float* weights,
                                 hipStream_t st) {
  return k <= 16 ? launch_route_type<TYPE, 1>(logits, T, E, k, scoring, ids, weights, st)
                 : launch_route_type<TYPE, 4>(logits, T, E, k, scoring, ids, weights, st);
}

hipError_t launch_route(const void* logits, int64_t T, int E, int k, int type, int scoring, int* ids, float* weights,
                        hipStream_t st) {
  // a launch holds fewer than 2^32 threads, up to 64 of them a token
  constexpr int64_t kLaunchTokens = int64_t(1) << 24;
  for (int64_t t = 0; t < T; t += kLaunchTokens) {
    const int64_t n = T - t < kLaunchTokens ? T - t : kLaunchTokens;
    const void* l = (const char*)logits + t * E * type_bytes(type);
    const hipError_t rc = type == kTypeF32 ? launch_route_k<kTypeF32>(l, n, E, k, scoring, ids + t * k, weights + t * k, st)
                          : type == kTypeF16
                              ? launch_route_k<kTypeF16>(l, n, E, k, scoring, ids + t * k, weights + t * k, st)
                              : launch_route_k<kTypeBf16>(l, n, E, k, scoring, ids + t * k, weights + t * k, st);
    if (rc != hipSuccess) return rc;
  }
  return hipSuccess;
}

hipError_t launch_plan(const RoutePlan& p, hipStream_t st) {
  const int blocks = p.ids && p.P >= kPlanSplit ? kPlanBlocks : 1;
  plan_kernel<<<blocks, kPlanThreads, 0, st>>>(p);
  return hipGetLastError();
}

hipError_t launch_combine(const float* part, const int* ids, const float* weights, const uint16_t* res, int64_t T,
                          int k, int E, int N, int64_t ld, int type, int out_type, void* out, hipStream_t st) {
  const bool wide = N % 4 == 0 && ld % 4 == 0 && (uintptr_t)out % (4 * type_bytes(out_type)) == 0;
  // a launch holds fewer than 2^32 threads: tokens of 2^30 at a time
  const int64_t per = wide ? N / 4 : N, tokens = std::max<int64_t>((int64_t(1) << 30) / per, 1);
  for (int64_t t = 0; t < T; t += tokens) {
    const int64_t n = std::min(tokens, T - t);
    const dim3 grid((unsigned)((n * per + 255) / 256));
    const float* p = part + t * k * N;
    const uint16_t* r = res ? res + t * ld : nullptr;
    void* o = (char*)out + t * ld * type_bytes(out_type);
    if (wide)
      combine_kernel<4><<<grid, 256, 0, st>>>(p, ids + t * k, weights + t * k, r, n, k, E, N, ld, type, out_type, o);
    else
      combine_kernel<1><<<grid, 256, 0, st>>>(p, ids + t * k, weights + t * k, r, n, k, E, N, ld, type, out_type, o);
  }
  return hipGetLastError();
}

}  // namespace swq
