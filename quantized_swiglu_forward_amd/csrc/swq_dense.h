// Internal interface between the host code and the kernels of the products
// with 16-bit weights, the 8-bit activation checkpoints, the SwiGLU with
// checkpoints and the router's loss and gradient.
#pragma once

#include "swq_mx4.h"

namespace swq {

// Activations of a product's epilogue (values fixed by the public header).
enum : int { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActGeluTanh = 4 };

// How the inner index r of an operand runs: along its rows (element p of row ...
// at p * ld + r) or down its columns (r * ld + p).
enum : int { kAlong = 0, kDown = 1 };

// out[p, q] = act(sum_r a(p, r) b(q, r) + bias[q]) + res[p, q]; the argument of act also to
// z (in the operands' type, or with z_scales as an 8-bit checkpoint).  p < P, q < Q, r < R.
struct DenseGemm {
  const uint16_t* a;
  const uint16_t* b;
  int64_t lda, ldb;
  int way_a, way_b;         // kAlong, kDown
  int64_t P, Q, R;
  int type;                 // the operands', the bias's, the residual's and z's 16-bit type
  int act;
  const uint16_t* bias;     // [Q] or null
  const uint16_t* res;      // [P, Q] or null
  void* out;                // [P, Q]
  int out_type;
  void* z;                  // [P, Q] or null
  uint8_t* z_scales;        // [P, ceil(Q / 32)]: z as a checkpoint; or null
  // set by plan_dense_gemm
  int kind;                 // kernel and tile shape
  int splits;               // blocks that share a tile's inner indexes, split_len each (a multiple of 64)
  int64_t split_len;
  int64_t part_ld;
  float* parts;             // with splits > 1: their sums [splits][P][part_ld], dense_parts_bytes
};
// The operands of a planned product that takes whole units: rows of 16-byte units from 16-byte aligned bases, lda and ldb
// multiples of 8, elements past R in a row's last unit zeros.
inline bool dense_takes_units(const DenseGemm& g) { return g.kind != 0; }
inline int64_t ceil8(int64_t n) { return (n + 7) / 8 * 8; }
// (false: no launch can hold it)
bool plan_dense_gemm(DenseGemm& g);
int64_t dense_parts_bytes(const DenseGemm& g);
hipError_t launch_dense_gemm(const DenseGemm& g, hipStream_t st);

// The gradients of one product in one launch: x (Along, Down), w (Down, Down), both plain, and the sums of n_sums
// partial sums [n_sums][N] (0: none).  Its blocks are set by plan_dense_pair.
struct DensePair {
  DenseGemm x, w;
  int x_blocks, w_blocks, w_first;
  int n_sums;
  const float* sums;
  int64_t N;
  uint16_t* dbias;
};
bool plan_dense_pair(DensePair& d, bool with_x, bool with_w);
hipError_t launch_dense_pair(const DensePair& d, int type, hipStream_t st);

// A tensor [R, K] in 16 bits, or with scales as an 8-bit checkpoint (K / 32 scales a row, rounded up).
struct Kept {
  const void* data;
  const uint8_t* scales;
};

hipError_t launch_mx8_quantize(const void* x, int64_t R, int64_t K, int type, void* codes, uint8_t* scales,
                               hipStream_t st);
hipError_t launch_mx8_dequantize(const void* codes, const uint8_t* scales, int64_t R, int64_t K, int type, void* out,
                                 hipStream_t st);

// hidden = silu(gate) up, with gate and up as checkpoints where the codes are not null
hipError_t launch_swiglu(const uint16_t* gate, const uint16_t* up, int64_t R, int64_t K, int type, uint16_t* hidden,
                         void* gcodes, uint8_t* gscales, void* ucodes, uint8_t* uscales, hipStream_t st);
hipError_t launch_swiglu_backward(const uint16_t* dhidden, Kept gate, Kept up, int64_t R, int64_t K, int type,
                                  uint16_t* dgate, uint16_t* dup, uint16_t* hidden, hipStream_t st);

// What a product's operands need first, in one launch: rows of 16-byte units, and dz.
struct PrepRows {           // src [R, K] (with scales a checkpoint) to rows of ceil8(K), zeros behind
  const void* src;
  const uint8_t* scales;
  int64_t R, K;
  uint16_t* dst;            // null: nothing to do
};
struct Prep {
  PrepRows rows[2];
  // dz = dout act'(z) [M, N], rows ceil8(N) apart with zeros behind (null: not wanted), and the sums of its columns:
  // act_parts(M, N) partial ones [..][N] in float32, or where that is 1 dbias itself (both null: not wanted)
  const uint16_t* dout;     // null: nothing to do
  Kept z;
  int64_t M, N;
  int act;
  uint16_t* dz;
  float* sums;
  uint16_t* dbias;
};
int64_t act_parts(int64_t M, int64_t N);
hipError_t launch_prep(const Prep& p, int type, hipStream_t st);
hipError_t launch_zero16(uint16_t* p, int64_t n, hipStream_t st);

// The router's balance loss (parts: balance_workspace bytes) and the gradient of its logits.
int64_t balance_workspace(int64_t T, int E);
hipError_t launch_balance(const void* logits, const int* ids, int64_t T, int E, int k, int type, int scoring,
                          float* loss, int* counts, float* slopes, void* parts, hipStream_t st);
hipError_t launch_route_backward(const void* logits, const int* ids, const float* dweights, const float* slopes,
                                 const float* dloss, int64_t T, int E, int k, int type, int scoring, void* dlogits,
                                 hipStream_t st);

}  // namespace swq
