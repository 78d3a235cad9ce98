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
#include "swq_mx4_device.h"

namespace swq {
namespace {

enum : int { kRouteSoftmax = 0, kRouteSoftmaxChosen = 1, kRouteSigmoid = 2, kRouteSigmoidChosen = 3 };

constexpr float kMaxFloat = 3.402823466e38f, kMinusInf = -__builtin_huge_valf();

// A logit as the router takes it: NaN ranks as -inf (masked), +inf as the largest float32.
template <int TYPE>
__device__ __forceinline__ float logit_at(const void* logits, int64_t at) {
  float v;
  if constexpr (TYPE == kTypeF32) v = ((const float*)logits)[at];
  else v = from_16(((const uint16_t*)logits)[at], TYPE);
  return v != v ? kMinusInf : fminf(v, kMaxFloat);
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
  return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v = fmaxf(v, __shfl_xor(v, d));
  return v;
}

// e^min(v, 0 or more) / (1 + e^-|v|) times e^-from: the sigmoid without underflow next to the row's largest
__device__ __forceinline__ float sigmoid_term(float v, float from) {
  return expf(fminf(v, 0.0f) - from) / (1.0f + expf(-fabsf(v)));
}

// p of a token's experts lane, lane + 64, ...; a row with nothing but -inf has p = 0.
template <int R>
__device__ __forceinline__ void shares(const float (&v)[R], bool sigmoid, float (&p)[R]) {
  float top = kMinusInf;
#pragma unroll
  for (int i = 0; i < R; ++i) top = fmaxf(top, v[i]);
  top = wave_max(top);
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    p[i] = v[i] == kMinusInf ? 0.0f : sigmoid ? sigmoid_term(v[i], fminf(top, 0.0f)) : expf(v[i] - top);
    sum += p[i];
  }
  sum = wave_sum(sum);
  const float by = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
  for (int i = 0; i < R; ++i) p[i] *= by;
}

// A wave per token: the sums of its tokens' p in registers, the counts in LDS.  parts: [blocks][E] sums, then
// [blocks][E + 1] counts, the last the tokens with a slot.
template <int TYPE, int R>
__global__ __launch_bounds__(256) void balance_kernel(const void* __restrict__ logits, const int* __restrict__ ids,
                                                      int64_t T, int E, int k, int scoring, int64_t rows,
                                                      float* __restrict__ sums, int* __restrict__ counts) {
  __shared__ int hist[64 * R + 1];
  __shared__ float part[4][64 * R];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#ifdef SWQ_LDS_POISON
  lds_poison(hist, sizeof(hist), kPoisonExp);
  lds_poison(part, sizeof(part), kPoisonFloat);
  __syncthreads();
#endif
  for (int e = threadIdx.x; e <= 64 * R; e += 256) hist[e] = 0;
  __syncthreads();
  float acc[R] = {};
  const int64_t t0 = (int64_t)blockIdx.x * rows, t1 = min(t0 + rows, T);
  for (int64_t t = t0 + wave; t < t1; t += 4) {
    const int id = lane < k ? ids[t * k + lane] : -1;
    const bool valid = id >= 0 && id < E;
    if (valid) atomicAdd(&hist[id], 1);
    if (!__ballot(valid)) continue;
    if (lane == 0) atomicAdd(&hist[64 * R], 1);
    float v[R], p[R];
#pragma unroll
    for (int i = 0; i < R; ++i) v[i] = 64 * i + lane < E ? logit_at<TYPE>(logits, t * E + 64 * i + lane) : kMinusInf;
    shares<R>(v, scoring >= kRouteSigmoid, p);
#pragma unroll
    for (int i = 0; i < R; ++i) acc[i] += p[i];
  }
#pragma unroll
  for (int i = 0; i < R; ++i) part[wave][64 * i + lane] = acc[i];
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += 256) {
    sums[(int64_t)blockIdx.x * E + e] = part[0][e] + part[1][e] + part[2][e] + part[3][e];
    counts[(int64_t)blockIdx.x * (E + 1) + e] = hist[e];
  }
  if (threadIdx.x == 0) counts[(int64_t)blockIdx.x * (E + 1) + E] = hist[64 * R];
}

__global__ __launch_bounds__(1024) void balance_join_kernel(const float* __restrict__ sums,
                                                            const int* __restrict__ part_counts, int blocks, int E,
                                                            float* __restrict__ loss, int* __restrict__ counts,
                                                            float* __restrict__ slopes) {
  __shared__ double all[1024];
  __shared__ int64_t number[1024];
  const int e = threadIdx.x;
  double sum = 0.0;
  int count = 0, tokens = 0;
  for (int b = 0; b < blocks; ++b) {
    if (e < E) sum += sums[(int64_t)b * E + e], count += part_counts[(int64_t)b * (E + 1) + e];
    tokens += part_counts[(int64_t)b * (E + 1) + E];
  }
  all[e] = sum * (double)count;
  number[e] = count;
  __syncthreads();
  for (int d = 512; d; d >>= 1) {
    if (e < d) all[e] += all[e + d], number[e] += number[e + d];
    __syncthreads();
  }
  const double by = number[0] ? (double)E / ((double)number[0] * (double)tokens) : 0.0;
  if (e < E) counts[e] = count, slopes[e] = (float)(by * (double)count);
  if (e == 0) *loss = (float)(by * all[0]);
}

// A wave per token; lane j has slot j, lane l the experts l, l + 64, ...
template <int TYPE, int R>
__global__ __launch_bounds__(256) void route_backward_kernel(const void* __restrict__ logits,
                                                             const int* __restrict__ ids,
                                                             const float* __restrict__ dweights,
                                                             const float* __restrict__ slopes,
                                                             const float* __restrict__ dloss, int64_t T, int E, int k,
                                                             int scoring, void* __restrict__ dlogits) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= T) return;
  const bool sigmoid = scoring >= kRouteSigmoid;
  const int id = lane < k ? ids[t * k + lane] : -1;
  const bool valid = id >= 0 && id < E;
  const bool any = __ballot(valid) != 0;
  float v[R], p[R], g[R];
#pragma unroll
  for (int i = 0; i < R; ++i) v[i] = 64 * i + lane < E ? logit_at<TYPE>(logits, t * E + 64 * i + lane) : kMinusInf;
  shares<R>(v, sigmoid, p);
  const float by = slopes && any ? dloss ? *dloss : 1.0f : 0.0f;
#pragma unroll
  for (int i = 0; i < R; ++i) g[i] = slopes && any && 64 * i + lane < E ? by * slopes[64 * i + lane] : 0.0f;
  // what a slot adds: of softmax to the derivative by p, else to the gradient itself
  const float dw = valid && dweights ? dweights[t * k + lane] : 0.0f;
  const float lv = valid ? logit_at<TYPE>(logits, t * E + id) : kMinusInf;
  float slot = dw;
  if (scoring != kRouteSoftmax) {
    const float top = wave_max(lv);
    float w = lv == kMinusInf ? 0.0f : scoring == kRouteSoftmaxChosen ? expf(lv - top)
              : sigmoid_term(lv, scoring == kRouteSigmoidChosen ? fminf(top, 0.0f) : 0.0f);
    if (scoring == kRouteSigmoid) {
      slot = dw * w * sigmoid_term(-lv, 0.0f);
    } else {
      const float sum = wave_sum(w);
      w = sum > 0.0f ? w / sum : 0.0f;
      slot = w * (dw - wave_sum(w * dw));
      if (scoring == kRouteSigmoidChosen) slot *= sigmoid_term(-lv, 0.0f);
    }
    if (lv == kMinusInf) slot = 0.0f;
  }
  float extra[R] = {};
  for (int j = 0; j < k; ++j) {
    const int e = __shfl(id, j);
    const float s = __shfl(slot, j);
#pragma unroll
    for (int i = 0; i < R; ++i) extra[i] += e == 64 * i + lane ? s : 0.0f;
  }
  if (scoring == kRouteSoftmax) {
#pragma unroll
    for (int i = 0; i < R; ++i) g[i] += extra[i], extra[i] = 0.0f;
  }
  float dot = 0.0f;
#pragma unroll
  for (int i = 0; i < R; ++i) dot += g[i] * p[i];
  dot = wave_sum(dot);
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if (64 * i + lane >= E) continue;
    float d = p[i] * (g[i] - dot);
    if (sigmoid) d *= v[i] == kMinusInf ? 0.0f : sigmoid_term(-v[i], 0.0f);
    d += extra[i];
    const int64_t at = t * E + 64 * i + lane;
    if constexpr (TYPE == kTypeF32) ((float*)dlogits)[at] = d;
    else ((uint16_t*)dlogits)[at] = to_16(d, TYPE);
  }
}

int64_t balance_rows(int64_t T) { return std::max<int64_t>(16, (T + 511) / 512); }

template <class F>
void by_experts(int E, F f) {
  if (E <= 64) f.template operator()<1>();
  else if (E <= 128) f.template operator()<2>();
  else if (E <= 256) f.template operator()<4>();
  else if (E <= 512) f.template operator()<8>();
  else f.template operator()<16>();
}

}  // namespace

int64_t balance_workspace(int64_t T, int E) {
  const int64_t blocks = (T + balance_rows(T) - 1) / balance_rows(T);
  return blocks * (2 * (int64_t)E + 1) * 4;
}

hipError_t launch_balance(const void* logits, const int* ids, int64_t T, int E, int k, int type, int scoring,
                          float* loss, int* counts, float* slopes, void* parts, hipStream_t st) {
  const int64_t rows = balance_rows(T);
  const int blocks = (int)((T + rows - 1) / rows);
  float* sums = (float*)parts;
  int* part_counts = (int*)(sums + (int64_t)blocks * E);
  if (blocks) {
    by_experts(E, [&]<int R>() {
      const auto kernel = type == kTypeF32 ? balance_kernel<kTypeF32, R>
                          : type == kTypeF16 ? balance_kernel<kTypeF16, R> : balance_kernel<kTypeBf16, R>;
      kernel<<<blocks, 256, 0, st>>>(logits, ids, T, E, k, scoring, rows, sums, part_counts);
    });
  }
  balance_join_kernel<<<1, 1024, 0, st>>>(sums, part_counts, blocks, E, loss, counts, slopes);
  return hipGetLastError();
}

hipError_t launch_route_backward(const void* logits, const int* ids, const float* dweights, const float* slopes,
                                 const float* dloss, int64_t T, int E, int k, int type, int scoring, void* dlogits,
                                 hipStream_t st) {
  constexpr int64_t kLaunchTokens = int64_t(1) << 24;     // a launch holds fewer than 2^32 threads
  by_experts(E, [&]<int R>() {
    const auto kernel = type == kTypeF32 ? route_backward_kernel<kTypeF32, R>
                        : type == kTypeF16 ? route_backward_kernel<kTypeF16, R> : route_backward_kernel<kTypeBf16, R>;
    for (int64_t t = 0; t < T; t += kLaunchTokens) {
      const int64_t n = std::min(kLaunchTokens, T - t);
      kernel<<<(unsigned)((n + 3) / 4), 256, 0, st>>>((const char*)logits + t * E * type_bytes(type), ids + t * k,
                                                      dweights ? dweights + t * k : nullptr, slopes, dloss, n, E, k,
                                                      scoring, (char*)dlogits + t * E * type_bytes(type));
    }
  });
  return hipGetLastError();
}

}  // namespace swq
