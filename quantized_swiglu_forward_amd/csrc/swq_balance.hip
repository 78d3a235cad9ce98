// The router's balance loss with the experts' counts, and the gradient of its logits.
//
// c_e: slots of expert e; N = sum c_e; T' = tokens with a slot; p_te: softmax over the experts, or for the sigmoid
// scorings sigma_te / sum_e sigma_te; P_e = sum over these tokens p_te / T'.
//   loss = E sum_e (c_e / N) P_e        slopes_e = E c_e / (N T'), the derivative by p_te
// (without a slot: 0).  The gradient of the logits, v_te = dloss slopes_e:
//   softmax        p_e (v_e - sum v p)           sigmoid   (1 - sigma_e) p_e (v_e - sum v p)
// and of the routing weights w_j of the slots j with expert e, d_j = dw_j:
//   softmax        p_e (sum_{j of e} d_j - sum_j d_j p_j), with v the same formula
//   of the chosen  w_j (d_j - sum d w)           sigmoid   d_j s_j (1 - s_j)
//   sigmoid of the chosen   (1 - s_j) w_j (d_j - sum d w)
#include <algorithm>

#include "swq_dense.h"
#include "swq_dense_device.h"

namespace swq {
namespace {

enum : int { kRouteSoftmax = 0, kRouteSoftmaxChosen = 1, kRouteSigmoid = 2, kRouteSigmoidChosen = 3 };

constexpr float kMaxFloat = 3.402823466e38f, kMinusInf = -__builtin_huge_valf();

// A logit as the router takes it: NaN ranks as -inf (masked), +inf as the largest float32.
__device__ __forceinline__ float as_logit(float v) { return v != v ? kMinusInf : fminf(v, kMaxFloat); }
template <int TYPE>
__device__ __forceinline__ float logit_at(const void* logits, int64_t at) {
  if constexpr (TYPE == kTypeF32) return as_logit(((const float*)logits)[at]);
  else return as_logit(from_16(((const uint16_t*)logits)[at], TYPE));
}

// G lanes per token, 16 or the wave, lane l with the R experts from l R on, four at a time (at any address).  Where all
// lanes have R of them there are no branches, each of which would wait for the loads before it.
template <int TYPE>
__device__ __forceinline__ void load4(const void* x, int64_t at, float* v) {
  if constexpr (TYPE == kTypeF32) {
    const u32x4 w = *(const u32x4_any*)((const float*)x + at);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = __uint_as_float(w[j]);
  } else {
    const u32x2 w = *(const u32x2_any*)((const uint16_t*)x + at);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = from_16((uint16_t)(w[j >> 1] >> (16 * (j & 1))), TYPE);
  }
}
template <int TYPE>
__device__ __forceinline__ void store4(void* x, int64_t at, const float* v) {
  if constexpr (TYPE == kTypeF32)
    *(u32x4_any*)((float*)x + at) = __builtin_bit_cast(u32x4, (f32x4){v[0], v[1], v[2], v[3]});
  else
    *(u32x2_any*)((uint16_t*)x + at) = (u32x2){pack16<TYPE>(v[0], v[1]), pack16<TYPE>(v[2], v[3])};
}
template <int TYPE, int G, int R>
__device__ __forceinline__ void load_row(const void* x, int64_t row, int first, int E, float rest, float (&v)[R]) {
  if (E == G * R) {
#pragma unroll
    for (int i = 0; i < R; i += 4) load4<TYPE>(x, row + first + i, v + i);
    return;
  }
#pragma unroll
  for (int i = 0; i < R; i += 4) {
    const int n = E - first - i;
    if (n >= 4) {
      load4<TYPE>(x, row + first + i, v + i);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[i + j] = rest;
        if (j < n) v[i + j] = TYPE == kTypeF32 ? ((const float*)x)[row + first + i + j]
                                               : from_16(((const uint16_t*)x)[row + first + i + j], TYPE);
      }
    }
  }
}
template <int TYPE, int G, int R>
__device__ __forceinline__ void load_logits(const void* logits, int64_t row, int first, int E, float (&v)[R]) {
  load_row<TYPE, G, R>(logits, row, first, E, kMinusInf, v);
#pragma unroll
  for (int i = 0; i < R; ++i) v[i] = as_logit(v[i]);
}

// op over a group of G lanes (16 neighbours by rotations of the row, or the wave); every lane gets the result.
template <int ROT>
__device__ __forceinline__ float rotate16(float v) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), 0x120 + ROT, 0xF, 0xF, true));
}
// op over the two rows of 16 lanes of a half, over the two halves
template <class Op>
__device__ __forceinline__ float across16(float v, Op op) {
  const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return op(__uint_as_float(p[0]), __uint_as_float(p[1]));
}
template <class Op>
__device__ __forceinline__ float across32(float v, Op op) {
  const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return op(__uint_as_float(p[0]), __uint_as_float(p[1]));
}
template <int G, class Op>
__device__ __forceinline__ float over_group(float v, Op op) {
  v = op(v, rotate16<8>(v));
  v = op(v, rotate16<4>(v));
  v = op(v, rotate16<2>(v));
  v = op(v, rotate16<1>(v));
  if constexpr (G == 64) {
    v = across16(v, op);
    v = across32(v, op);
  }
  return v;
}
template <int G>
__device__ __forceinline__ float group_sum(float v) {
  return over_group<G>(v, [](float a, float b) { return a + b; });
}
template <int G>
__device__ __forceinline__ float group_max(float v) {
  return over_group<G>(v, [](float a, float b) { return fmaxf(a, b); });
}

// e^t for t <= 0 (the hardware's exp2: off by 2^-23 and the argument's rounding, t 2^-24 of itself)
__device__ __forceinline__ float exp_down(float t) { return __builtin_amdgcn_exp2f(t * 1.4426950408889634f); }

// The largest of a row, to be taken from its logits (never -inf, which would be -inf less -inf).
__device__ __forceinline__ float from_top(float top) { return fmaxf(top, -kMaxFloat); }

// sigma(v) e^-from: the sigmoid without underflow next to the row's largest (from = that where it is below 0); 0 for -inf
__device__ __forceinline__ float sigmoid_term(float v, float from) {
  const float e = exp_down(-fabsf(v)), up = v < 0.0f ? e : 1.0f;
  return (from < 0.0f ? exp_down(fminf(v, 0.0f) - from) : up) * __builtin_amdgcn_rcpf(1.0f + e);
}
__device__ __forceinline__ float sigmoid(float v) {
  const float e = exp_down(-fabsf(v));
  return (v < 0.0f ? e : 1.0f) * __builtin_amdgcn_rcpf(1.0f + e);
}

// p of a token's experts; a row with nothing but -inf has p = 0.
template <int G, int R, bool SIGMOID>
__device__ __forceinline__ void shares(const float (&v)[R], float (&p)[R]) {
  float top = v[0];
#pragma unroll
  for (int i = 1; i < R; ++i) top = fmaxf(top, v[i]);
  top = from_top(group_max<G>(top));
  float sum = 0.0f;
  if (SIGMOID && !__any(top < 0.0f)) {         // (the wave's rows all have a logit from 0 on)
#pragma unroll
    for (int i = 0; i < R; ++i) p[i] = sigmoid(v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < R; ++i) p[i] = SIGMOID ? sigmoid_term(v[i], fminf(top, 0.0f)) : exp_down(v[i] - top);
  }
#pragma unroll
  for (int i = 0; i < R; ++i) sum += p[i];
  sum = group_sum<G>(sum);
  const float by = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
  for (int i = 0; i < R; ++i) p[i] *= by;
}

// A token's slots: lane l has the slots l, l + G, ...
template <int G, int KR>
__device__ __forceinline__ bool load_ids(const int* ids, int64_t t, int k, int E, int lane, int (&id)[KR]) {
  bool any = false;
#pragma unroll
  for (int s = 0; s < KR; ++s) {
    id[s] = lane + G * s < k ? ids[t * k + lane + G * s] : -1;
    if (id[s] >= E) id[s] = -1;
    any |= id[s] >= 0;
  }
  return group_max<G>(any ? 1.0f : 0.0f) > 0.0f;
}

// The sum over the block of a double each; every thread gets it.  `meet` has 16 entries.
template <int ROT>
__device__ __forceinline__ double rotate16_double(double v) {
  const u32x2 w = __builtin_bit_cast(u32x2, v);
  return __builtin_bit_cast(double, (u32x2){(uint32_t)__builtin_amdgcn_update_dpp(0, (int)w[0], 0x120 + ROT, 0xF, 0xF, true),
                                            (uint32_t)__builtin_amdgcn_update_dpp(0, (int)w[1], 0x120 + ROT, 0xF, 0xF, true)});
}
__device__ __forceinline__ double block_sum(double v, double* meet) {
  v += rotate16_double<8>(v);
  v += rotate16_double<4>(v);
  v += rotate16_double<2>(v);
  v += rotate16_double<1>(v);
  v += __shfl_xor(v, 16);
  v += __shfl_xor(v, 32);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) meet[threadIdx.x >> 6] = v;
  __syncthreads();
  double all = 0.0;
  for (int w = 0; w < (int)blockDim.x >> 6; ++w) all += meet[w];
  return all;
}

// A block sums the p and counts the slots of `rows` tokens, its groups of lanes in turn: sums in registers, then over
// the block through LDS, counts in LDS (integers, so that no order matters).  Its sums go to
// sums[block][pitch], its counts to counts[block][pitch], its slots and tokens with a slot to totals[block][2]; a
// block that is alone concludes.  Latency bounds it, a row's loads and reductions: 8192 x 256 (4.5 MB) takes 5.6 us and
// its join 5.2 to 6.0; 65 x 64, alone, 4.5.  Atomics on float sums would have needed cleared memory and an order.
template <int TYPE, int G, int R, int KR, bool SIGMOID, int THREADS>
__global__ __launch_bounds__(THREADS) void balance_kernel(const void* __restrict__ logits, const int* __restrict__ ids,
                                                          int64_t T, int E, int k, int64_t rows, int pitch,
                                                          float* __restrict__ sums, int* __restrict__ counts,
                                                          int* __restrict__ totals, float* __restrict__ loss,
                                                          int* __restrict__ out_counts, float* __restrict__ slopes) {
  constexpr int GROUPS = THREADS / G, WAVES = THREADS / 64, EX = G * R;
  __shared__ int hist[EX + 1];
  __shared__ float part[WAVES][EX];
  __shared__ double meet[16];
  const int lane = threadIdx.x & (G - 1), group = threadIdx.x / G, wave = threadIdx.x >> 6;
#ifdef SWQ_LDS_POISON
  lds_poison(hist, sizeof(hist), kPoisonExp);
  lds_poison(part, sizeof(part), kPoisonFloat);
  lds_poison(meet, sizeof(meet), kPoisonFloat);
  __syncthreads();
#endif
  for (int e = threadIdx.x; e <= EX; e += THREADS) hist[e] = 0;
  __syncthreads();
  float acc[R] = {};
  const int64_t t0 = (int64_t)blockIdx.x * rows, t1 = min(t0 + rows, T);
  for (int64_t t = t0 + group; t < t1; t += GROUPS) {
    float v[R], p[R];
    int id[KR];
    const bool live = load_ids<G, KR>(ids, t, k, E, lane, id);
    load_logits<TYPE, G, R>(logits, t * E, lane * R, E, v);
#pragma unroll
    for (int s = 0; s < KR; ++s)
      if (id[s] >= 0) atomicAdd(&hist[id[s]], 1);
    if (lane == 0 && live) atomicAdd(&hist[EX], 1);
    shares<G, R, SIGMOID>(v, p);
#pragma unroll
    for (int i = 0; i < R; ++i) acc[i] += live ? p[i] : 0.0f;
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if constexpr (G == 16) {
      const auto add = [](float a, float b) { return a + b; };
      acc[i] = across32(across16(acc[i], add), add);
    }
    if ((threadIdx.x & 63) < G) part[wave][lane * R + i] = acc[i];
  }
  __syncthreads();
  const auto sum_of = [&](int e) SWQ_INLINE {
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) sum += part[w][e];
    return sum;
  };
  const int e = threadIdx.x;                 // (E <= 2 THREADS)
  double slots = 0.0;
  for (int i = e; i < E; i += THREADS) slots += hist[i];
  slots = block_sum(slots, meet);
  if (gridDim.x == 1) {
    const int tokens = hist[EX];
    const double by = tokens ? (double)E / (slots * (double)tokens) : 0.0;
    double all = 0.0;
    for (int i = e; i < E; i += THREADS) {
      const double count = hist[i];
      all += (double)sum_of(i) * count;
      out_counts[i] = hist[i];
      slopes[i] = (float)(by * count);
    }
    all = block_sum(all, meet);
    if (e == 0) *loss = (float)(by * all);
    return;
  }
  for (int i = e; i < E; i += THREADS) {
    sums[(int64_t)blockIdx.x * pitch + i] = sum_of(i);
    counts[(int64_t)blockIdx.x * pitch + i] = hist[i];
  }
  if (e == 0) {
    totals[2 * blockIdx.x] = (int)slots;
    totals[2 * blockIdx.x + 1] = hist[EX];
    if (blockIdx.x == 0) totals[2 * gridDim.x] = 0;          // the ticket of the join
  }
}

// 32 experts per block, a thread with four of them and a slice of the blocks' sums (one block for all of them took 7.1 to 8.8 us:
// a CU alone draws the 512 KB that long).  The block that is last by the
// ticket adds the blocks' parts of the loss, in their order.
constexpr int kJoinExperts = 32, kJoinThreads = 256;
__global__ __launch_bounds__(kJoinThreads) void balance_join_kernel(const float* __restrict__ sums,
                                                                    const int* __restrict__ part_counts, int* totals,
                                                                    double* parts, int blocks, int E, int pitch,
                                                                    float* __restrict__ loss, int* __restrict__ counts,
                                                                    float* __restrict__ slopes) {
  constexpr int SLICES = kJoinThreads / 8, WAVES = kJoinThreads / 64;
  __shared__ __attribute__((aligned(16))) float psum[SLICES][kJoinExperts];
  __shared__ __attribute__((aligned(16))) int pcount[SLICES][kJoinExperts];
  __shared__ int total[WAVES][2];
#ifdef SWQ_LDS_POISON
  lds_poison(psum, sizeof(psum), kPoisonFloat);
  lds_poison(pcount, sizeof(pcount), kPoisonExp);
  lds_poison(total, sizeof(total), kPoisonExp);
  __syncthreads();
#endif
  const int quad = threadIdx.x & 7, slice = threadIdx.x >> 3, e0 = blockIdx.x * kJoinExperts;
  int slots = 0, tokens = 0;                 // (kJoinThreads >= blocks; T k < 2^31)
  if ((int)threadIdx.x < blocks) slots = totals[2 * threadIdx.x], tokens = totals[2 * threadIdx.x + 1];
  f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
  i32x4 n = {0, 0, 0, 0};
  if (e0 + 4 * quad < E) {
#pragma unroll 8
    for (int b = slice; b < blocks; b += SLICES) {
      s += *(const f32x4*)(sums + (int64_t)b * pitch + e0 + 4 * quad);
      n += *(const i32x4*)(part_counts + (int64_t)b * pitch + e0 + 4 * quad);
    }
  }
  *(f32x4*)&psum[slice][4 * quad] = s;
  *(i32x4*)&pcount[slice][4 * quad] = n;
#pragma unroll
  for (int d = 32; d; d >>= 1) slots += __shfl_xor(slots, d), tokens += __shfl_xor(tokens, d);
  if ((threadIdx.x & 63) == 0) total[threadIdx.x >> 6][0] = slots, total[threadIdx.x >> 6][1] = tokens;
  __syncthreads();
  if (threadIdx.x >= 64) return;             // the first wave has an expert per lane
  slots = tokens = 0;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) slots += total[w][0], tokens += total[w][1];
  const double by = tokens ? (double)E / ((double)slots * (double)tokens) : 0.0;
  double all = 0.0;
  const int e = e0 + threadIdx.x;
  if (threadIdx.x < kJoinExperts && e < E) {
    double sum = 0.0;
    int count = 0;
#pragma unroll
    for (int i = 0; i < SLICES; ++i) sum += (double)psum[i][threadIdx.x], count += pcount[i][threadIdx.x];
    counts[e] = count;
    slopes[e] = (float)(by * (double)count);
    all = sum * (double)count;
  }
  all += rotate16_double<8>(all);
  all += rotate16_double<4>(all);
  all += rotate16_double<2>(all);
  all += rotate16_double<1>(all);
  all += __shfl_xor(all, 16);
  if (threadIdx.x) return;
  if (gridDim.x > 1) {
    __hip_atomic_store(&parts[blockIdx.x], all, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (__hip_atomic_fetch_add(&totals[2 * blocks], 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) !=
        (int)gridDim.x - 1)
      return;
    all = 0.0;
#pragma unroll 8
    for (int b = 0; b < (int)gridDim.x; ++b)
      all += __hip_atomic_load(&parts[b], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  *loss = (float)(by * all);
}

// The gradient, G lanes per token as above; slot j is in lane j % G.  One reading of logits and ids and one writing:
// 8192 x 256 bf16, top 8, 5.9 to 7.5 us (8.9 MB, a launch's 2.5 and one round of dependent loads and reductions); 65 x 64 3.8.
template <int TYPE, int G, int R, int KR, bool SIGMOID>
__global__ __launch_bounds__(256) void route_backward_kernel(const void* __restrict__ logits,
                                                             const int* __restrict__ ids,
                                                             const float* __restrict__ dweights,
                                                             const float* __restrict__ slopes,
                                                             const float* __restrict__ dloss, int64_t T, int E, int k,
                                                             int scoring, void* __restrict__ dlogits) {
  const int lane = threadIdx.x & (G - 1);
  const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) / G, t = min(at, T - 1);
  // (no lane leaves early: the reductions take every lane of their group)
  float v[R], p[R], g[R], extra[R];
  int id[KR];
  const bool live = load_ids<G, KR>(ids, t, k, E, lane, id);
  load_logits<TYPE, G, R>(logits, t * E, lane * R, E, v);
  float dw[KR], lv[KR], slot[KR];
#pragma unroll
  for (int s = 0; s < KR; ++s) {
    dw[s] = id[s] >= 0 && dweights ? dweights[t * k + lane + G * s] : 0.0f;
    lv[s] = id[s] >= 0 ? logit_at<TYPE>(logits, t * E + id[s]) : kMinusInf;
    dw[s] = lv[s] == kMinusInf ? 0.0f : dw[s];           // (a masked expert's weight is 0, whatever stands in its dweights)
    slot[s] = dw[s];
  }
#pragma unroll
  for (int i = 0; i < R; ++i) g[i] = 0.0f;
  if (slopes) {
    const float by = live ? dloss ? *dloss : 1.0f : 0.0f;        // (slopes of no expert are 0)
    load_row<kTypeF32, G, R>(slopes, 0, lane * R, E, 0.0f, g);
#pragma unroll
    for (int i = 0; i < R; ++i) g[i] *= by;
  }
  shares<G, R, SIGMOID>(v, p);
  // what a slot adds: of softmax to the derivative by p, else to the gradient itself
  if (scoring != kRouteSoftmax) {
    float top = kMinusInf, w[KR], sum = 0.0f, dot = 0.0f;
#pragma unroll
    for (int s = 0; s < KR; ++s) top = fmaxf(top, lv[s]);
    top = from_top(group_max<G>(top));
    const float from = scoring == kRouteSigmoidChosen ? fminf(top, 0.0f) : 0.0f;
#pragma unroll
    for (int s = 0; s < KR; ++s) {
      w[s] = SIGMOID ? sigmoid_term(lv[s], from) : exp_down(lv[s] - top);
      sum += w[s];
    }
    if (scoring != kRouteSigmoid) {
      sum = group_sum<G>(sum);
      const float per = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
      for (int s = 0; s < KR; ++s) w[s] *= per, dot += w[s] * dw[s];
      dot = group_sum<G>(dot);
    }
#pragma unroll
    for (int s = 0; s < KR; ++s) {
      slot[s] = w[s] * (dw[s] - dot);
      if (SIGMOID) slot[s] *= sigmoid(-lv[s]);
    }
  }
#pragma unroll
  for (int i = 0; i < R; ++i) extra[i] = 0.0f;
  if (dweights) {
    // a lane first finds the slots of its experts, then adds them one by one, in the slots' order: as many rounds as one lane has
#pragma unroll
    for (int s = 0; s < KR; ++s) {
      const int most = min(G, k - G * s);
      uint64_t mine = 0;
      for (int j = 0; j < most; ++j) mine |= (uint64_t)((uint32_t)(__shfl(id[s], j, G) - lane * R) < (uint32_t)R) << j;
      while (__ballot(mine != 0)) {
        const int j = mine ? __builtin_ctzll(mine) : 0;
        const int e = __shfl(id[s], j, G) - lane * R;
        const float add = __shfl(slot[s], j, G);
#pragma unroll
        for (int i = 0; i < R; ++i) extra[i] += mine && e == i ? add : 0.0f;
        mine &= mine - 1;
      }
    }
  }
  if (scoring == kRouteSoftmax) {
#pragma unroll
    for (int i = 0; i < R; ++i) g[i] += extra[i], extra[i] = 0.0f;
  }
  float dot = 0.0f;
#pragma unroll
  for (int i = 0; i < R; ++i) dot += g[i] * p[i];
  dot = group_sum<G>(dot);
  if (at >= T) return;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    float d = p[i] * (g[i] - dot);
    if (SIGMOID) d *= sigmoid(-v[i]);
    p[i] = d + extra[i];
  }
  const int64_t o = t * E + lane * R;
  if (E == G * R) {
#pragma unroll
    for (int i = 0; i < R; i += 4) store4<TYPE>(dlogits, o + i, p + i);
    return;
  }
#pragma unroll
  for (int i = 0; i < R; i += 4) {
    const int n = E - lane * R - i;
    if (n >= 4) {
      store4<TYPE>(dlogits, o + i, p + i);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (j >= n) continue;
        if constexpr (TYPE == kTypeF32) ((float*)dlogits)[o + i + j] = p[i + j];
        else ((uint16_t*)dlogits)[o + i + j] = to_16(p[i + j], TYPE);
      }
    }
  }
}

// f.operator()<TYPE, G, R, KR, SIGMOID>() for the type, the numbers of experts and slots and the scoring: sixteen lanes
// up to 256 experts, the wave from there on.
template <int TYPE, bool SIGMOID, class F>
void by_sizes(int E, int k, F f) {
  if (E <= 256) {
    const auto with = [&]<int R>() {
      if (k <= 16) f.template operator()<TYPE, 16, R, 1, SIGMOID>();
      else f.template operator()<TYPE, 16, R, 4, SIGMOID>();
    };
    if (E <= 64) with.template operator()<4>();
    else if (E <= 128) with.template operator()<8>();
    else with.template operator()<16>();
  } else if (E <= 512) {
    f.template operator()<TYPE, 64, 8, 1, SIGMOID>();
  } else {
    f.template operator()<TYPE, 64, 16, 1, SIGMOID>();
  }
}
template <class F>
void by_shape(int type, int E, int k, int scoring, F f) {
  const auto with = [&]<int TYPE>() {
    if (scoring >= kRouteSigmoid) by_sizes<TYPE, true>(E, k, f);
    else by_sizes<TYPE, false>(E, k, f);
  };
  if (type == kTypeF32) with.template operator()<kTypeF32>();
  else if (type == kTypeF16) with.template operator()<kTypeF16>();
  else with.template operator()<kTypeBf16>();
}

// Tokens of a block: up to 128 tokens one block of 1024 threads does it all, saving the join's launch; else at most 256
// blocks of 512 threads (with the join 10.1 us at 8192 x 256 and 21 at 65536 x 256; 128 blocks of 1024 took 10.6 and 25).
constexpr int64_t kAlone = 128;
int64_t balance_rows(int64_t T) { return T <= kAlone ? kAlone : std::max<int64_t>(32, (T + 255) / 256); }
int balance_pitch(int E) { return (E + 3) / 4 * 4; }

}  // namespace

int64_t balance_workspace(int64_t T, int E) {
  const int64_t blocks = (T + balance_rows(T) - 1) / balance_rows(T);
  return T > kAlone ? 32 * 8 + blocks * (balance_pitch(E) * 8 + 8) + 4 : 0;
}

hipError_t launch_balance(const void* logits, const int* ids, int64_t T, int E, int k, int type, int scoring,
                          float* loss, int* counts, float* slopes, void* ws, hipStream_t st) {
  const int64_t rows = balance_rows(T);
  const int blocks = std::max(1, (int)((T + rows - 1) / rows)), pitch = balance_pitch(E);   // (no tokens: one block, zeros)
  double* parts = (double*)ws;                                  // [E / 32]
  float* sums = (float*)(parts + 32);                           // [blocks][pitch]
  int* part_counts = (int*)(sums + (int64_t)blocks * pitch);    // [blocks][pitch]
  int* totals = part_counts + (int64_t)blocks * pitch;          // [blocks][2], the ticket
  by_shape(type, E, k, scoring, [&]<int TYPE, int G, int R, int KR, bool SIGMOID>() {
    if (blocks == 1)
      balance_kernel<TYPE, G, R, KR, SIGMOID, 1024><<<1, 1024, 0, st>>>(
          logits, ids, T, E, k, rows, pitch, sums, part_counts, totals, loss, counts, slopes);
    else
      balance_kernel<TYPE, G, R, KR, SIGMOID, 512><<<blocks, 512, 0, st>>>(
          logits, ids, T, E, k, rows, pitch, sums, part_counts, totals, loss, counts, slopes);
  });
  if (blocks > 1)
    balance_join_kernel<<<(E + kJoinExperts - 1) / kJoinExperts, kJoinThreads, 0, st>>>(
        sums, part_counts, totals, parts, blocks, E, pitch, loss, counts, slopes);
  return hipGetLastError();
}

hipError_t launch_route_backward(const void* logits, const int* ids, const float* dweights, const float* slopes,
                                 const float* dloss, int64_t T, int E, int k, int type, int scoring, void* dlogits,
                                 hipStream_t st) {
  constexpr int64_t kLaunchTokens = int64_t(1) << 24;     // a launch holds fewer than 2^32 threads
  by_shape(type, E, k, scoring, [&]<int TYPE, int G, int R, int KR, bool SIGMOID>() {
    for (int64_t t = 0; t < T; t += kLaunchTokens) {
      const int64_t n = std::min(kLaunchTokens, T - t);
      route_backward_kernel<TYPE, G, R, KR, SIGMOID><<<(unsigned)((n * G + 255) / 256), 256, 0, st>>>(
          (const char*)logits + t * E * type_bytes(type), ids + t * k, dweights ? dweights + t * k : nullptr, slopes,
          dloss, n, E, k, scoring, (char*)dlogits + t * E * type_bytes(type));
    }
  });
  return hipGetLastError();
}

}  // namespace swq
