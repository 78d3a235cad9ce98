// Internal interface between the host code and the kernels of the microscaled
// 4-bit (MXFP4) operators, the router and the experts' MLP.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace swq {

// Element types (values fixed by the public header).
enum : int { kTypeBf16 = 0, kTypeF32 = 1, kTypeF16 = 2 };
inline int type_bytes(int t) { return t == kTypeF32 ? 4 : 2; }

// Where a product's rows of x come from:
//   kXBf16   bf16 rows
//   kXF16    binary16 rows, split into two bf16 operands by the kernel
//   kXPlanes two bf16 rows (hi, lo), `plane` elements apart
enum : int { kXBf16 = 0, kXF16 = 1, kXPlanes = 2 };

// Kernels of a product with MXFP4 weights.
enum : int { kFew, kSmallTiles, kMidTiles, kLargeTiles };

// Most experts whose offsets the products read themselves (one per lane of a wave).
constexpr int kOffsetExperts = 64;

// One tile of rows of a grouped product.
struct RowTile {
  int expert;   // -1: rows of no expert, written as zeros
  int first;    // first slot (row of the sorted order)
  int rows;     // 1 .. tile height
  int pad;
};

// out[row(slot), n] = sum_k x[xrow(slot), k] w[expert(slot)][n, k], or with w2 the
// SwiGLU of two such sums.  Dense products: tiles null, one expert, rows = M.
struct MxGemm {
  const uint16_t* x;
  int64_t plane;            // kXPlanes: elements between the two planes
  const uint32_t* w;        // codes [E][N][K/8]
  const uint8_t* s;         // scales [E][N][K/32]
  const uint32_t* w2;       // the up matrix, or null
  const uint8_t* s2;
  const uint16_t* res;      // residual [rows, N] in x's type, or null
  void* out;                // [rows, N] in out_type; SwiGLU with hidden_planes: bf16 planes
  int64_t out_plane;        // elements between the planes of a split hidden tensor
  int rows, K, N, E;
  int64_t wrows;            // rows of W from one expert to the next (N, or more where the product takes some columns)
  int xsrc;                 // kXBf16, kXF16, kXPlanes
  const int* xperm;         // slot -> row (x row: that / xdiv), or null: slot s reads x row s
  int xdiv;
  int xrows;                // rows of x behind xperm
  int vec;                  // rows of out and the residual allow accesses of 4 (1) or of 4 and 8 (2) outputs
  int type;                 // x's and the residual's 16-bit type
  int out_type;
  int hidden_planes;        // 1: write the hidden tensor as two bf16 planes
  const RowTile* tiles;     // tile table, or null
  const int* ntiles;
  const int* offsets;       // without a table: [E + 1] the experts' first rows, E <= 64, or null
  const int* perm;          // slot -> row of out, or null (the same)
  int max_tiles;            // with tiles or offsets: the most there can be; else 0
  int check_only;           // 1: the launch functions launch nothing and say whether one launch can hold the product
  int kind;                 // kFew .. kLargeTiles (mx4_gemm_kind)
  int splits;               // K splits (mx4_gemm_splits; 0 and 1: none) and their partial sums [splits][rows][N]
  float* parts;
  int split_chunks;         // chunks of 128 inputs per split (set by the launch)
  const int* ids;           // without tiles: the expert of every row (few rows, taken one by one), or null

#ifdef __HIPCC__
  // the parts of an output's way to memory that this product has
  __device__ uint16_t* low_plane() const { return hidden_planes ? (uint16_t*)out + out_plane : nullptr; }
  __device__ int stride() const { return N; }                 // from one output row to the next
  __device__ void add_residual(float* f, int64_t at) const;   // eight neighbours, 16-byte aligned
  __device__ void add_one(float& f, int64_t at) const;
#endif
};

// out[m, n] = sum_k a[m, k] w[n, k] of two MXFP4 operands; rows of out are ld apart (N, or more
// where the launch takes some columns).
struct Mx4Matmul {
  const uint32_t* a;
  const uint8_t* sa;
  const uint32_t* w;
  const uint8_t* s;
  void* out;
  int M, K, N, ld, out_type;
  int vec;                  // as MxGemm

#ifdef __HIPCC__
  __device__ uint16_t* low_plane() const { return nullptr; }
  __device__ int stride() const { return ld; }
  __device__ void add_residual(float*, int64_t) const {}
  __device__ void add_one(float&, int64_t) const {}
#endif
};

struct RoutePlan {
  const int* ids;           // [P] expert of each row, or null
  const int* offsets;       // [E + 1] sorted rows' first slots, or null
  int P, E, tile;           // rows, experts, tile height
  RowTile* tiles;           // out
  int* ntiles;              // out
  int* perm;                // out (ids only)
};
// Most tiles a plan of P rows and E experts can have.
inline int64_t max_row_tiles(int64_t P, int64_t E, int tile) {
  return P / tile + (E + 2 < P ? E + 2 : P) + 1;
}

hipError_t launch_mx4_quantize(const void* x, int64_t blocks, int type, uint32_t* codes, uint8_t* scales,
                               hipStream_t st);
hipError_t launch_mx4_dequantize(const uint32_t* codes, const uint8_t* scales, int64_t blocks, int type, void* out,
                                 hipStream_t st);
// binary16 rows [n] to two bf16 planes, n a multiple of 8
hipError_t launch_mx4_split(const uint16_t* x, int64_t n, uint16_t* planes, int64_t plane, hipStream_t st);
hipError_t launch_mx4_gemm(const MxGemm& p, hipStream_t st);
// The kernel for a product (MxGemm::kind); one choice for products that share a plan.
int mx4_gemm_kind(const MxGemm& p);
int mx4_gemm_splits(const MxGemm& p);
int mx4_gemm_tile(const MxGemm& p);           // row tile height of its kind, for the plan
bool mx4_gemm_takes_planes(const MxGemm& p);  // its kind wants binary16 x as planes
// out[t] = res[t] + sum_j weights[t, j] x[t k + j] W[ids[t k + j]]^T for few tokens (p.rows = tokens k)
hipError_t launch_mx4_down(const MxGemm& p, const float* weights, int k, hipStream_t st);
// bytes of workspace that the product of two MXFP4 matrices takes (0: none)
int64_t mx4_matmul_workspace(const Mx4Matmul& p);
hipError_t launch_mx4_matmul(const Mx4Matmul& p, void* ws, hipStream_t st);
hipError_t launch_route(const void* logits, int64_t T, int E, int k, int type, int scoring, int* ids, float* weights,
                        hipStream_t st);
hipError_t launch_plan(const RoutePlan& p, hipStream_t st);
// out[t] = residual[t] + sum_j weights[t, j] part[t k + j] over the slots whose id is an expert
// (part has rows of N; res and out rows of ld, from their first column on)
hipError_t launch_combine(const float* part, const int* ids, const float* weights, const uint16_t* res, int64_t T,
                          int k, int E, int N, int64_t ld, int type, int out_type, void* out, hipStream_t st);

// Compute units of the current device (swq_api.hip).
int device_cus();
// The library's per-(device, stream) buffers (swq_api.hip).
int stream_workspace(hipStream_t stream, size_t need, void** out, int slot);

}  // namespace swq
