// The router's choice, the order of a product grouped by expert, and the sum
// over a token's experts.
#include "swq_mx4.h"
#include "swq_mx4_device.h"

namespace swq {
namespace {

// Routing weights (values fixed by the public header).
enum : int { kRouteSoftmax = 0, kRouteSoftmaxChosen = 1, kRouteSigmoid = 2, kRouteSigmoidChosen = 3 };

constexpr int kMaxExperts = 1024;

__device__ __forceinline__ float load_logit(const void* p, int64_t at, int type) {
  const float v = type == kTypeF32 ? ((const float*)p)[at] : from_16(((const uint16_t*)p)[at], type);
  // NaN ranks below everything; +inf counts as the largest float32
  return v != v ? -__builtin_inff() : fminf(v, 3.402823466e38f);
}

// A chosen logit's weight before the division by the sum: e^(v - top), or the sigmoid
// e^min(v, 0) / (1 + e^-|v|), over the chosen ones times e^-min(top, 0), so that
// very low logits do not make it 0 / 0.
__device__ __forceinline__ float routing_term(float v, float top, int scoring) {
  if (scoring <= kRouteSoftmaxChosen) return expf(v - top);
  const float from = scoring == kRouteSigmoidChosen ? fminf(top, 0.0f) : 0.0f;
  return expf(fminf(v, 0.0f) - from) / (1.0f + expf(-fabsf(v)));
}

// One wave per token.  A logit and its index make one 64-bit key that orders
// by value, then by the lower index: k rounds of a maximum over the wave.
__global__ __launch_bounds__(256) void route_kernel(const void* __restrict__ logits, int64_t T, int E, int k, int type,
                                                    int scoring, int* __restrict__ ids, float* __restrict__ weights) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= T) return;
  constexpr int R = kMaxExperts / 64;
  float v[R];
#pragma unroll
  for (int i = 0; i < R; ++i) v[i] = 64 * i + lane < E ? load_logit(logits, t * E + 64 * i + lane, type) : -__builtin_inff();
  float top = -__builtin_inff(), sum = 0.0f;
  const bool over_all = scoring == kRouteSoftmax;
  if (over_all) {
#pragma unroll
    for (int i = 0; i < R; ++i) top = fmaxf(top, v[i]);
    for (int d = 32; d; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
#pragma unroll
    for (int i = 0; i < R; ++i) sum += v[i] > -__builtin_inff() ? expf(v[i] - top) : 0.0f;
    for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d);
  }
  int my_id = -1;
  float my_w = 0.0f, chosen = 0.0f;
  uint32_t used = 0;
  for (int j = 0; j < k; ++j) {
    float bv = -__builtin_inff();
    int bi = kMaxExperts;
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (!(used >> i & 1) && v[i] > bv) bv = v[i], bi = 64 * i + lane;
    for (int d = 32; d; d >>= 1) {
      const float ov = __shfl_xor(bv, d);
      const int oi = __shfl_xor(bi, d);
      if (ov > bv || (ov == bv && oi < bi)) bv = ov, bi = oi;
    }
    if (bi == kMaxExperts) break;              // only -inf is left
    if ((bi & 63) == lane) used |= 1u << (bi >> 6);
    if (j == 0) top = bv;
    const float w = routing_term(bv, top, scoring);
    chosen += w;
    if (lane == j) my_id = bi, my_w = w;
  }
  if (lane < k) {
    const float by = over_all ? sum : scoring == kRouteSigmoid ? 1.0f : chosen;
    ids[t * k + lane] = my_id;
    weights[t * k + lane] = my_id < 0 ? 0.0f : my_w / by;
  }
}

// Order of the rows of a grouped product and its tiles, in one block.  With
// ids: the slots of each expert's rows (their order within an expert decides
// no result: every output row depends on its own input row alone).  With
// offsets: the groups as given, made non-decreasing and cut at P; the rows
// before the first and after the last group become tiles of no expert.
// Thread t holds expert t.
constexpr int kPlanThreads = 1024, kPlanAhead = 8;

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
  const int t = threadIdx.x;
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
  for (int i = 0; i < tiles; ++i)
    p.tiles[tile_end - tiles + i] = RowTile{t, first + i * p.tile, min(p.tile, rows - i * p.tile), 0};
  if (p.ids) {
    if (t == kPlanThreads - 1) *p.ntiles = tile_end;
    if (t < p.E) next[t] = first;
    __syncthreads();
    for (int i0 = t; i0 < p.P; i0 += kPlanThreads * kPlanAhead) {
      int e[kPlanAhead];
#pragma unroll
      for (int j = 0; j < kPlanAhead; ++j) e[j] = i0 + j * kPlanThreads < p.P ? p.ids[i0 + j * kPlanThreads] : -1;
#pragma unroll
      for (int j = 0; j < kPlanAhead; ++j)
        if (e[j] >= 0 && e[j] < p.E) p.perm[atomicAdd(&next[e[j]], 1)] = i0 + j * kPlanThreads;
    }
  } else if (t == kPlanThreads - 1) {          // rows of no expert, before and after the groups
    int n = tile_end;
    for (int i = 0; i < next[0]; i += p.tile) p.tiles[n++] = RowTile{-1, i, min(p.tile, next[0] - i), 0};
    for (int i = last; i < p.P; i += p.tile) p.tiles[n++] = RowTile{-1, i, min(p.tile, p.P - i), 0};
    *p.ntiles = n;
  }
}

// One thread per V neighbours of an output row: the k partial rows are read four slots
// at a time, each slot's id and weight first.
template <int V>
__global__ __launch_bounds__(256) void combine_kernel(const float* __restrict__ part, const int* __restrict__ ids,
                                                      const float* __restrict__ weights,
                                                      const uint16_t* __restrict__ res, int64_t T, int k, int E, int N,
                                                      int type, int out_type, void* __restrict__ out) {
  const int per = N / V;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t t = i / per;
  const int n = (int)(i - t * per) * V;
  if (t >= T) return;
  const int64_t at = t * N + n;
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

hipError_t launch_route(const void* logits, int64_t T, int E, int k, int type, int scoring, int* ids, float* weights,
                        hipStream_t st) {
  route_kernel<<<dim3((unsigned)((T + 3) / 4)), 256, 0, st>>>(logits, T, E, k, type, scoring, ids, weights);
  return hipGetLastError();
}

hipError_t launch_plan(const RoutePlan& p, hipStream_t st) {
  plan_kernel<<<1, kPlanThreads, 0, st>>>(p);
  return hipGetLastError();
}

hipError_t launch_combine(const float* part, const int* ids, const float* weights, const uint16_t* res, int64_t T,
                          int k, int E, int N, int type, int out_type, void* out, hipStream_t st) {
  const bool wide = N % 4 == 0 && (uintptr_t)out % (4 * type_bytes(out_type)) == 0;
  const int64_t threads = T * (wide ? N / 4 : N);
  if ((threads + 255) / 256 >= (1LL << 31)) return hipErrorInvalidValue;
  const dim3 grid((unsigned)((threads + 255) / 256));
  if (wide) combine_kernel<4><<<grid, 256, 0, st>>>(part, ids, weights, res, T, k, E, N, type, out_type, out);
  else combine_kernel<1><<<grid, 256, 0, st>>>(part, ids, weights, res, T, k, E, N, type, out_type, out);
  return hipGetLastError();
}

}  // namespace swq
