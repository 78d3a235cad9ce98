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

// G lanes per token, 16 or the wave, lane l with the R experts from l R on, four at a time (at any address).
template <int TYPE, int R>
__device__ __forceinline__ void load_logits(const void* logits, int64_t row, int first, int E, float (&v)[R]) {
#pragma unroll
  for (int i = 0; i < R; i += 4) {
    const int n = E - first - i;
    if (n >= 4) {
      if constexpr (TYPE == kTypeF32) {
        const u32x4 w = *(const u32x4_any*)((const float*)logits + row + first + i);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[i + j] = as_logit(__uint_as_float(w[j]));
      } else {
        const u32x2 w = *(const u32x2_any*)((const uint16_t*)logits + row + first + i);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[i + j] = as_logit(from_16((uint16_t)(w[j >> 1] >> (16 * (j & 1))), TYPE));
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[i + j] = j < n ? logit_at<TYPE>(logits, row + first + i + j) : kMinusInf;
    }
  }
}

template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int d = G / 2; d; d >>= 1) v += __shfl_xor(v, d);
  return v;
}
template <int G>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int d = G / 2; d; d >>= 1) v = fmaxf(v, __shfl_xor(v, d));
  return v;
}

// sigma(v) e^-from: the sigmoid without underflow next to the row's largest (from = that, or 0)
__device__ __forceinline__ float sigmoid_term(float v, float from) {
  return expf(fminf(v, 0.0f) - from) / (1.0f + expf(-fabsf(v)));
}

// p of a token's experts; a row with nothing but -inf has p = 0.
template <int G, int R>
__device__ __forceinline__ void shares(const float (&v)[R], bool sigmoid, float (&p)[R]) {
  float top = kMinusInf;
#pragma unroll
  for (int i = 0; i < R; ++i) top = fmaxf(top, v[i]);
  top = group_max<G>(top);
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    p[i] = v[i] == kMinusInf ? 0.0f : sigmoid ? sigmoid_term(v[i], fminf(top, 0.0f)) : expf(v[i] - top);
    sum += p[i];
  }
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

// The loss, counts and slopes from the sums over all tokens, by the block: thread e < E has expert e's.
__device__ __forceinline__ void conclude(double sum, int count, int64_t tokens, int E, double* all, int64_t* number,
                                         float* loss, int* counts, float* slopes) {
  const int e = threadIdx.x;
  all[e] = sum * (double)count;
  number[e] = count;
  __syncthreads();
  for (int d = blockDim.x / 2; d; d >>= 1) {
    if (e < d) all[e] += all[e + d], number[e] += number[e + d];
    __syncthreads();
  }
  const double by = number[0] ? (double)E / ((double)number[0] * (double)tokens) : 0.0;
  if (e < E) counts[e] = count, slopes[e] = (float)(by * (double)count);
  if (e == 0) *loss = (float)(by * all[0]);
}

// A block sums the p and counts the slots of `rows` tokens, its 1024 / G groups of lanes in turn: sums in
// registers, then over the block through LDS, counts in LDS (integers, so that no order matters).  Its sums go to
// sums[block][pitch], its counts to counts[block][pitch], the tokens with a slot at E; a block that is alone concludes.
//
// Two launches' latency: 8192 tokens of 256 (4.3 MB) 128 blocks and the join.
template <int TYPE, int G, int R, int KR>
__global__ __launch_bounds__(1024) void balance_kernel(const void* __restrict__ logits, const int* __restrict__ ids,
                                                       int64_t T, int E, int k, int scoring, int64_t rows, int pitch,
                                                       float* __restrict__ sums, int* __restrict__ counts,
                                                       float* __restrict__ loss, int* __restrict__ out_counts,
                                                       float* __restrict__ slopes) {
  constexpr int GROUPS = 1024 / G, EX = G * R;
  __shared__ int hist[EX + 1];
  __shared__ float part[16][EX];
  __shared__ double all[1024];
  __shared__ int64_t number[1024];
  const int lane = threadIdx.x & (G - 1), group = threadIdx.x / G, wave = threadIdx.x >> 6;
#ifdef SWQ_LDS_POISON
  lds_poison(hist, sizeof(hist), kPoisonExp);
  lds_poison(part, sizeof(part), kPoisonFloat);
  lds_poison(all, sizeof(all), kPoisonFloat);
  lds_poison(number, sizeof(number), kPoisonExp);
  __syncthreads();
#endif
  for (int e = threadIdx.x; e <= EX; e += 1024) hist[e] = 0;
  __syncthreads();
  float acc[R] = {};
  const int64_t t0 = (int64_t)blockIdx.x * rows, t1 = min(t0 + rows, T);
  for (int64_t t = t0 + group; t < t1; t += GROUPS) {
    float v[R], p[R];
    int id[KR];
    load_logits<TYPE, R>(logits, t * E, lane * R, E, v);
    const bool live = load_ids<G, KR>(ids, t, k, E, lane, id);
#pragma unroll
    for (int s = 0; s < KR; ++s)
      if (id[s] >= 0) atomicAdd(&hist[id[s]], 1);
    if (lane == 0 && live) atomicAdd(&hist[EX], 1);
    shares<G, R>(v, scoring >= kRouteSigmoid, p);
#pragma unroll
    for (int i = 0; i < R; ++i) acc[i] += live ? p[i] : 0.0f;
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if constexpr (G == 16) {
      acc[i] += __shfl_xor(acc[i], 16);
      acc[i] += __shfl_xor(acc[i], 32);
    }
    if ((threadIdx.x & 63) < G) part[wave][lane * R + i] = acc[i];
  }
  __syncthreads();
  const int e = threadIdx.x;
  float sum = 0.0f;
  if (e < EX) {
#pragma unroll
    for (int w = 0; w < 16; ++w) sum += part[w][e];
  }
  if (gridDim.x == 1) {
    conclude(e < E ? (double)sum : 0.0, e < E ? hist[e] : 0, hist[EX], E, all, number, loss, out_counts, slopes);
    return;
  }
  if (e < E) {
    sums[(int64_t)blockIdx.x * pitch + e] = sum;
    counts[(int64_t)blockIdx.x * pitch + e] = hist[e];
  }
  if (e == 0) counts[(int64_t)blockIdx.x * pitch + E] = hist[EX];
}

// Four experts (the count of the tokens after the last) and a slice of the blocks per thread; the slices' sums meet
// in LDS.
__global__ __launch_bounds__(1024) void balance_join_kernel(const float* __restrict__ sums,
                                                            const int* __restrict__ part_counts, int blocks, int E,
                                                            int pitch, float* __restrict__ loss,
                                                            int* __restrict__ counts, float* __restrict__ slopes) {
  __shared__ double psum[4][1024];
  __shared__ int pcount[4][1024];
  __shared__ double all[1024];
  __shared__ int64_t number[1024];
#ifdef SWQ_LDS_POISON
  lds_poison(psum, sizeof(psum), kPoisonFloat);
  lds_poison(pcount, sizeof(pcount), kPoisonExp);
  lds_poison(all, sizeof(all), kPoisonFloat);
  lds_poison(number, sizeof(number), kPoisonExp);
  __syncthreads();
#endif
  const int quads = pitch / 4, slices = 1024 / quads, quad = threadIdx.x % quads, slice = threadIdx.x / quads;
  double s[4] = {};
  int n[4] = {};
  if (slice < slices) {
#pragma unroll 8
    for (int b = slice; b < blocks; b += slices) {
      const f32x4 f = *(const f32x4*)(sums + (int64_t)b * pitch + 4 * quad);
      const i32x4 c = *(const i32x4*)(part_counts + (int64_t)b * pitch + 4 * quad);
#pragma unroll
      for (int j = 0; j < 4; ++j) s[j] += f[j], n[j] += c[j];
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) psum[j][threadIdx.x] = s[j], pcount[j][threadIdx.x] = n[j];
  __syncthreads();
  const auto total = [&](int e, double& sum, int& count) {
    sum = 0.0, count = 0;
    for (int i = 0; i < slices; ++i) sum += psum[e & 3][i * quads + e / 4], count += pcount[e & 3][i * quads + e / 4];
  };
  double sum = 0.0, unused;
  int count = 0, tokens;
  if ((int)threadIdx.x < E) total(threadIdx.x, sum, count);
  total(E, unused, tokens);
  conclude(sum, count, tokens, E, all, number, loss, counts, slopes);
}

// The gradient, G lanes per token as above; slot j is in lane j % G.
template <int TYPE, int G, int R, int KR>
__global__ __launch_bounds__(256) void route_backward_kernel(const void* __restrict__ logits,
                                                             const int* __restrict__ ids,
                                                             const float* __restrict__ dweights,
                                                             const float* __restrict__ slopes,
                                                             const float* __restrict__ dloss, int64_t T, int E, int k,
                                                             int scoring, void* __restrict__ dlogits) {
  const int lane = threadIdx.x & (G - 1);
  const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) / G, t = min(at, T - 1);
  // (no lane leaves early: the reductions take every lane of their group)
  const bool sigmoid = scoring >= kRouteSigmoid;
  float v[R], p[R], g[R], extra[R];
  int id[KR];
  load_logits<TYPE, R>(logits, t * E, lane * R, E, v);
  const bool live = load_ids<G, KR>(ids, t, k, E, lane, id);
  float dw[KR], lv[KR], slot[KR];
#pragma unroll
  for (int s = 0; s < KR; ++s) {
    dw[s] = id[s] >= 0 && dweights ? dweights[t * k + lane + G * s] : 0.0f;
    lv[s] = id[s] >= 0 ? logit_at<TYPE>(logits, t * E + id[s]) : kMinusInf;
    slot[s] = dw[s];
  }
  const float by = slopes && live ? dloss ? *dloss : 1.0f : 0.0f;
#pragma unroll
  for (int i = 0; i < R; ++i) g[i] = slopes && live && lane * R + i < E ? by * slopes[lane * R + i] : 0.0f;
  shares<G, R>(v, sigmoid, p);
  // what a slot adds: of softmax to the derivative by p, else to the gradient itself
  if (scoring != kRouteSoftmax) {
    float top = kMinusInf, w[KR], sum = 0.0f, dot = 0.0f;
#pragma unroll
    for (int s = 0; s < KR; ++s) top = fmaxf(top, lv[s]);
    top = group_max<G>(top);
    const float from = scoring == kRouteSigmoidChosen ? fminf(top, 0.0f) : 0.0f;
#pragma unroll
    for (int s = 0; s < KR; ++s) {
      w[s] = lv[s] == kMinusInf ? 0.0f : sigmoid ? sigmoid_term(lv[s], from) : expf(lv[s] - top);
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
      if (sigmoid) slot[s] *= lv[s] == kMinusInf ? 0.0f : sigmoid_term(-lv[s], 0.0f);
    }
  }
#pragma unroll
  for (int i = 0; i < R; ++i) extra[i] = 0.0f;
  if (dweights) {
#pragma unroll
    for (int s = 0; s < KR; ++s) {
      for (int j = 0; j < G && G * s + j < k; ++j) {
        const int e = __shfl(id[s], j, G) - lane * R;
        const float add = __shfl(slot[s], j, G);
#pragma unroll
        for (int i = 0; i < R; ++i) extra[i] += e == i ? add : 0.0f;
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
  for (int i = 0; i < R; i += 4) {
    float d[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      d[j] = p[i + j] * (g[i + j] - dot);
      if (sigmoid) d[j] *= v[i + j] == kMinusInf ? 0.0f : sigmoid_term(-v[i + j], 0.0f);
      d[j] += extra[i + j];
    }
    const int64_t o = t * E + lane * R + i;
    const int n = E - lane * R - i;
    if constexpr (TYPE == kTypeF32) {
      if (n >= 4) {
        *(u32x4_any*)((float*)dlogits + o) = __builtin_bit_cast(u32x4, (f32x4){d[0], d[1], d[2], d[3]});
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (j < n) ((float*)dlogits)[o + j] = d[j];
      }
    } else if (n >= 4) {
      *(u32x2_any*)((uint16_t*)dlogits + o) = (u32x2){pack16<TYPE>(d[0], d[1]), pack16<TYPE>(d[2], d[3])};
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < n) ((uint16_t*)dlogits)[o + j] = to_16(d[j], TYPE);
    }
  }
}

// f.operator()<TYPE, G, R, KR>() for the type and the numbers of experts and slots: sixteen lanes up to 256
// experts, the wave from there on.
template <int TYPE, class F>
void by_sizes(int E, int k, F f) {
  if (E <= 256) {
    const auto with = [&]<int R>() {
      if (k <= 16) f.template operator()<TYPE, 16, R, 1>();
      else f.template operator()<TYPE, 16, R, 4>();
    };
    if (E <= 64) with.template operator()<4>();
    else if (E <= 128) with.template operator()<8>();
    else with.template operator()<16>();
  } else if (E <= 512) {
    f.template operator()<TYPE, 64, 8, 1>();
  } else {
    f.template operator()<TYPE, 64, 16, 1>();
  }
}
template <class F>
void by_shape(int type, int E, int k, F f) {
  if (type == kTypeF32) by_sizes<kTypeF32>(E, k, f);
  else if (type == kTypeF16) by_sizes<kTypeF16>(E, k, f);
  else by_sizes<kTypeBf16>(E, k, f);
}

// Tokens of a block: up to 128 tokens one block does it all, saving the join's launch.
int64_t balance_rows(int64_t T) { return T <= 128 ? 128 : std::max<int64_t>(64, (T + 255) / 256); }
int balance_pitch(int E) { return (E + 1 + 3) / 4 * 4; }

}  // namespace

int64_t balance_workspace(int64_t T, int E) {
  const int64_t blocks = (T + balance_rows(T) - 1) / balance_rows(T);
  return blocks > 1 ? blocks * balance_pitch(E) * 8 : 0;
}

hipError_t launch_balance(const void* logits, const int* ids, int64_t T, int E, int k, int type, int scoring,
                          float* loss, int* counts, float* slopes, void* parts, hipStream_t st) {
  const int64_t rows = balance_rows(T);
  const int blocks = std::max(1, (int)((T + rows - 1) / rows)), pitch = balance_pitch(E);   // (no tokens: one block, zeros)
  float* sums = (float*)parts;
  int* part_counts = (int*)(sums + (int64_t)blocks * pitch);
  by_shape(type, E, k, [&]<int TYPE, int G, int R, int KR>() {
    balance_kernel<TYPE, G, R, KR><<<blocks, 1024, 0, st>>>(logits, ids, T, E, k, scoring, rows, pitch, sums,
                                                            part_counts, loss, counts, slopes);
  });
  if (blocks > 1)
    balance_join_kernel<<<1, 1024, 0, st>>>(sums, part_counts, blocks, E, pitch, loss, counts, slopes);
  return hipGetLastError();
}

hipError_t launch_route_backward(const void* logits, const int* ids, const float* dweights, const float* slopes,
                                 const float* dloss, int64_t T, int E, int k, int type, int scoring, void* dlogits,
                                 hipStream_t st) {
  constexpr int64_t kLaunchTokens = int64_t(1) << 24;     // a launch holds fewer than 2^32 threads
  by_shape(type, E, k, [&]<int TYPE, int G, int R, int KR>() {
    for (int64_t t = 0; t < T; t += kLaunchTokens) {
      const int64_t n = std::min(kLaunchTokens, T - t);
      route_backward_kernel<TYPE, G, R, KR><<<(unsigned)((n * G + 255) / 256), 256, 0, st>>>(
          (const char*)logits + t * E * type_bytes(type), ids + t * k, dweights ? dweights + t * k : nullptr, slopes,
          dloss, n, E, k, scoring, (char*)dlogits + t * E * type_bytes(type));
    }
  });
  return hipGetLastError();
}

}  // namespace swq
