// C-ABI entry points of the microscaled 4-bit (MXFP4) operators, the router
// and the experts' MLP (declared in include/swiglu_q.h): validation on the
// host, then launches on the caller's stream.
#include <algorithm>
#include <cmath>

#include "../../include/swiglu_q.h"
#include "swq_mx4.h"

using namespace swq;

namespace {

constexpr int kWsSlot = 2;            // the experts' workspace beside the MLP's two
// Whether the tokens' slots (T k of them) are taken one by one, each reading its expert's weights, or by expert.
// One by one saves the plan, a join and the few-row kernel's poorer reading, about 37.5 MB's worth and a fifth of
// the bytes of the experts reached; it pays for every expert that several tokens share, again.  The experts reached are
// reckoned for ids that spread evenly.  Measured, us one by one / by expert (columns: tokens):
//   k of E, H x I           2           3           4           5           6           8           12
//   8 of 64   2048 x 1024   20 / 31     28 / 36     33 / 43     41 / 45     45 / 53     58 / 57     82 / 67
//   8 of 256  2048 x 1024   20 / 31     28 / 37     32 / 45     42 / 53     46 / 57     59 / 69     85 / 89
//   4 of 16   2048 x 1024   14 / 23     19 / 29     21 / 29     26 / 29     28 / 29     34 / 30     47 / 30
//   4 of 4    2048 x 1024   12 / 21     17 / 21     19 / 21     24 / 21     26 / 21     33 / 21     46 / 31
//   8 of 8    2048 x 1024   19 / 24     27 / 24     31 / 25     40 / 24     43 / 24     56 / 25     78 / 34
//   2 of 8    4096 x 4096   33 / 45     45 / 55     59 / 59     70 / 65     83 / 65    105 / 64    154 / 73
//   4 of 32   2880 x 2880   31 / 44     40 / 47     51 / 64     59 / 66     71 / 74     89 / 89    123 / 108
// Past six tokens only many experts (256) or small ones (512 x 256: 7 / 15) still gain, and all go by expert.
constexpr int64_t kDirectTokens = 6;
bool slot_by_slot(int64_t T, int64_t k, int64_t E, int64_t H, int64_t I, int64_t Ho) {
  if (T > kDirectTokens) return false;
  const double expert = (2.0 * H * I + (double)I * Ho) * (0.5 + 1.0 / 32);      // bytes
  const double reached = E * (1 - std::pow(1 - std::min(1.0, (double)k / E), (double)T));
  return (T * k - reached) * expert <= 37.5e6 + 0.2 * reached * expert;
}
// The experts' float32 outputs that wait for their sum: what the 256 MB last-level cache still
// holds when the sum reads them (4096 tokens, 8 of 64 experts, 2048 columns, 268 MB: in one
// piece 529 us, in two 515, in three 558).  Equal pieces: 1280 and 768 columns, the least rounds of tiles
// over the CUs, took 528 where two of 1024 took 530.
constexpr int64_t kPartBytes = int64_t(160) << 20;
constexpr int64_t kMaxRows = int64_t(1) << 30, kMaxK = int64_t(1) << 20;

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }
bool type_ok(int t) { return t == SWQ_TYPE_BF16 || t == SWQ_TYPE_F32 || t == SWQ_TYPE_F16; }
bool type16_ok(int t) { return t == SWQ_TYPE_BF16 || t == SWQ_TYPE_F16; }
int64_t align256(int64_t v) { return (v + 255) / 256 * 256; }

// Shapes of one product: rows of x, inputs, outputs.
int check_shape(int64_t rows, int64_t K, int64_t N) {
  if (rows < 0 || K <= 0 || N <= 0) return SWQ_ERR_SHAPE;
  if (K % 32 != 0 || K > kMaxK || rows > kMaxRows || N > kMaxRows) return SWQ_ERR_SHAPE;
  // the kernels number their tiles in 31 bits
  if (((rows + 15) / 16 + 1024) * ((N + 15) / 16) >= (int64_t(1) << 31)) return SWQ_ERR_SHAPE;
  return SWQ_OK;
}

// A matrix of codes and scales: both there, the codes 16-byte aligned.
int check_codes(const uint32_t* W, const void* s) {
  if (!W || !s) return SWQ_ERR_NULL;
  return aligned(W, 16) ? SWQ_OK : SWQ_ERR_ALIGN;
}

int check_status(hipError_t e) { return e == hipSuccess ? SWQ_OK : SWQ_ERR_HIP; }

// Columns of the experts' outputs that are computed and summed at once.
int64_t part_columns(int64_t P, int64_t Ho) {
  const int64_t parts = (P * Ho * 4 + kPartBytes - 1) / kPartBytes;
  return ((Ho + parts - 1) / parts + 255) / 256 * 256;
}

// Bytes of a plan in the workspace: the tile count, the tile table, the order.
struct PlanLayout {
  int64_t tiles, perm, total;
};
PlanLayout plan_layout(int64_t P, int64_t E, int tile, bool with_perm) {
  PlanLayout l;
  l.tiles = 256;
  l.perm = l.tiles + align256(max_row_tiles(P, E, tile) * (int64_t)sizeof(RowTile));
  l.total = l.perm + (with_perm ? align256(P * 4) : 0);
  return l;
}

// Widths that N and the bases allow (MxGemm::vec).
int vec_ok(int64_t N, const void* out, const void* res, int out_type) {
  if (N % 8 == 0 && aligned(out, 16) && (!res || aligned(res, 16))) return 2;
  return N % 4 == 0 && aligned(out, 4 * type_bytes(out_type)) && (!res || aligned(res, 8));
}

// Whether a launch can hold the product (sizes, kind and tiles are set, pointers need not be).
bool fits(MxGemm g) {
  g.check_only = 1;
  return launch_mx4_gemm(g, nullptr) == hipSuccess;
}

// x as the product's kernels read it: binary16 rows become two bf16 planes in
// the workspace where they ask for it.
int64_t planes_bytes(const MxGemm& g, int64_t rows) {
  return g.xsrc == kXF16 && mx4_gemm_takes_planes(g) ? 2 * align256(rows * g.K * 2) : 0;
}
int to_planes(MxGemm& g, int64_t rows, void* ws, hipStream_t st) {
  if (!planes_bytes(g, rows)) return SWQ_OK;
  const int64_t plane = align256(rows * g.K * 2) / 2;
  const int rc = check_status(launch_mx4_split(g.x, rows * g.K, (uint16_t*)ws, plane, st));
  g.x = (const uint16_t*)ws;
  g.plane = plane;
  g.xsrc = kXPlanes;
  return rc;
}

// Order and tiles of g's rows; with ids, *perm is the order.
int run_plan(MxGemm& g, char* ws, const PlanLayout& l, const int* ids, const int* offsets, int tile, hipStream_t st,
             const int** perm = nullptr) {
  RoutePlan r{};
  r.ids = ids;
  r.offsets = offsets;
  r.P = g.rows;
  r.E = g.E;
  r.tile = tile;
  r.ntiles = (int*)ws;
  r.tiles = (RowTile*)(ws + l.tiles);
  r.perm = ids ? (int*)(ws + l.perm) : nullptr;
  if (perm) *perm = r.perm;
  g.tiles = r.tiles;
  g.ntiles = r.ntiles;
  return check_status(launch_plan(r, st));
}

}  // namespace

extern "C" {

int swiglu_q_mx4_quantize(const void* x, int64_t R, int64_t K, int type, uint32_t* codes, void* scales, void* stream) {
  if (!x || !codes || !scales) return SWQ_ERR_NULL;
  if (!type_ok(type)) return SWQ_ERR_UNSUPPORTED;
  if (R < 0 || K <= 0 || K % 32 != 0 || K > kMaxK || R > kMaxRows || R * K >= (int64_t(1) << 41)) return SWQ_ERR_SHAPE;
  if (!aligned(x, 16) || !aligned(codes, 16)) return SWQ_ERR_ALIGN;
  if (R == 0) return SWQ_OK;
  (void)hipGetLastError();
  return check_status(launch_mx4_quantize(x, R * (K / 32), type, codes, (uint8_t*)scales, (hipStream_t)stream));
}

int swiglu_q_mx4_dequantize(const uint32_t* codes, const void* scales, int64_t R, int64_t K, int type, void* out,
                            void* stream) {
  if (!codes || !scales || !out) return SWQ_ERR_NULL;
  if (!type_ok(type)) return SWQ_ERR_UNSUPPORTED;
  if (R < 0 || K <= 0 || K % 32 != 0 || K > kMaxK || R > kMaxRows || R * K >= (int64_t(1) << 41)) return SWQ_ERR_SHAPE;
  if (!aligned(codes, 16) || !aligned(out, 16)) return SWQ_ERR_ALIGN;
  if (R == 0) return SWQ_OK;
  (void)hipGetLastError();
  return check_status(
      launch_mx4_dequantize(codes, (const uint8_t*)scales, R * (K / 32), type, out, (hipStream_t)stream));
}

int swiglu_q_mx4_linear(const void* x, const uint32_t* W, const void* s, const void* residual, int64_t M, int64_t K,
                        int64_t N, int type, int out_mode, void* out, void* stream) {
  if (!x || !out) return SWQ_ERR_NULL;
  int rc = check_codes(W, s);
  if (rc != SWQ_OK) return rc;
  if (!type16_ok(type) || (out_mode != type && out_mode != SWQ_LINEAR_F32)) return SWQ_ERR_UNSUPPORTED;
  rc = check_shape(M, K, N);
  if (rc != SWQ_OK) return rc;
  if (!aligned(x, 16) || !aligned(out, type_bytes(out_mode)) || !aligned(residual, 2)) return SWQ_ERR_ALIGN;
  if (M == 0) return SWQ_OK;
  MxGemm g{};
  g.x = (const uint16_t*)x;
  g.w = W;
  g.s = (const uint8_t*)s;
  g.res = (const uint16_t*)residual;
  g.out = out;
  g.rows = (int)M;
  g.K = (int)K;
  g.N = (int)N;
  g.E = 1;
  g.wrows = N;
  g.xsrc = type == SWQ_TYPE_F16 ? kXF16 : kXBf16;
  g.xdiv = 1;
  g.type = type;
  g.out_type = out_mode;
  g.vec = vec_ok(N, out, residual, out_mode);
  g.kind = mx4_gemm_kind(g);
  g.splits = mx4_gemm_splits(g);
  if (!fits(g)) return SWQ_ERR_SHAPE;
  const int64_t planes = planes_bytes(g, M), parts = g.splits > 1 ? g.splits * M * N * 4 : 0;
  void* ws = nullptr;
  if (planes + parts) {
    rc = stream_workspace((hipStream_t)stream, (size_t)(planes + parts), &ws, kWsSlot);
    if (rc != SWQ_OK) return rc;
    g.parts = (float*)((char*)ws + planes);
  }
  (void)hipGetLastError();            // before the first launch: an error left by others is not this call's
  rc = to_planes(g, M, ws, (hipStream_t)stream);
  if (rc != SWQ_OK) return rc;
  return check_status(launch_mx4_gemm(g, (hipStream_t)stream));
}

int swiglu_q_mx4_matmul(const uint32_t* A, const void* sa, const uint32_t* W, const void* sw, int64_t M, int64_t K,
                        int64_t N, int out_mode, void* out, void* stream) {
  if (!out) return SWQ_ERR_NULL;
  int rc = check_codes(A, sa);
  if (rc != SWQ_OK) return rc;
  rc = check_codes(W, sw);
  if (rc != SWQ_OK) return rc;
  if (!type_ok(out_mode)) return SWQ_ERR_UNSUPPORTED;
  rc = check_shape(M, K, N);
  if (rc != SWQ_OK) return rc;
  if (!aligned(out, type_bytes(out_mode))) return SWQ_ERR_ALIGN;
  if (M == 0) return SWQ_OK;
  Mx4Matmul p{A, (const uint8_t*)sa, W, (const uint8_t*)sw, out, (int)M, (int)K, (int)N, (int)N, out_mode,
              vec_ok(N, out, nullptr, out_mode)};
  void* ws = nullptr;
  if (const int64_t need = mx4_matmul_workspace(p)) {
    rc = stream_workspace((hipStream_t)stream, (size_t)need, &ws, kWsSlot);
    if (rc != SWQ_OK) return rc;
  }
  (void)hipGetLastError();
  return check_status(launch_mx4_matmul(p, ws, (hipStream_t)stream));
}

int swiglu_q_mx4_grouped_linear(const void* x, const int32_t* offsets, const uint32_t* W, const void* s, int64_t P,
                                int64_t E, int64_t K, int64_t N, int type, int out_mode, void* out, void* stream_v) {
  hipStream_t stream = (hipStream_t)stream_v;
  if (!x || !offsets || !out) return SWQ_ERR_NULL;
  int rc = check_codes(W, s);
  if (rc != SWQ_OK) return rc;
  if (!type16_ok(type) || (out_mode != type && out_mode != SWQ_LINEAR_F32)) return SWQ_ERR_UNSUPPORTED;
  if (E < 1 || E > SWQ_MAX_EXPERTS) return SWQ_ERR_SHAPE;
  rc = check_shape(P, K, N);
  if (rc != SWQ_OK) return rc;
  if (!aligned(x, 16) || !aligned(offsets, 4) || !aligned(out, type_bytes(out_mode))) return SWQ_ERR_ALIGN;
  if (P == 0) return SWQ_OK;
  MxGemm g{};
  g.x = (const uint16_t*)x;
  g.w = W;
  g.s = (const uint8_t*)s;
  g.out = out;
  g.rows = (int)P;
  g.K = (int)K;
  g.N = (int)N;
  g.E = (int)E;
  g.wrows = N;
  g.xsrc = type == SWQ_TYPE_F16 ? kXF16 : kXBf16;
  g.xdiv = 1;
  g.type = type;
  g.out_type = out_mode;
  g.vec = vec_ok(N, out, nullptr, out_mode);
  g.kind = mx4_gemm_kind(g);
  const int tile = mx4_gemm_tile(g);
  const bool planned = E > kOffsetExperts;
  g.max_tiles = (int)max_row_tiles(P, E, tile);
  if (!fits(g)) return SWQ_ERR_SHAPE;
  const PlanLayout l = planned ? plan_layout(P, E, tile, false) : PlanLayout{0, 0, 0};
  void* ws = nullptr;
  if (const int64_t need = l.total + planes_bytes(g, P)) rc = stream_workspace(stream, (size_t)need, &ws, kWsSlot);
  if (rc != SWQ_OK) return rc;
  (void)hipGetLastError();
  if (planned) {
    rc = run_plan(g, (char*)ws, l, nullptr, offsets, tile, stream);
  } else {
    g.offsets = offsets;
  }
  if (rc == SWQ_OK) rc = to_planes(g, P, (char*)ws + l.total, stream);
  if (rc != SWQ_OK) return rc;
  return check_status(launch_mx4_gemm(g, stream));
}

int swiglu_q_route(const void* logits, int64_t T, int64_t E, int k, int type, int scoring, int32_t* ids,
                   float* weights, void* stream) {
  if (!logits || !ids || !weights) return SWQ_ERR_NULL;
  if (!type_ok(type) || scoring < SWQ_ROUTE_SOFTMAX || scoring > SWQ_ROUTE_SIGMOID_CHOSEN) return SWQ_ERR_UNSUPPORTED;
  if (T < 0 || T > kMaxRows || E < 1 || E > SWQ_MAX_EXPERTS || k < 1 || k > SWQ_MAX_CHOSEN || k > E)
    return SWQ_ERR_SHAPE;
  if (!aligned(logits, type_bytes(type)) || !aligned(ids, 4) || !aligned(weights, 4)) return SWQ_ERR_ALIGN;
  if (T == 0) return SWQ_OK;
  (void)hipGetLastError();
  return check_status(launch_route(logits, T, (int)E, k, type, scoring, ids, weights, (hipStream_t)stream));
}

int swiglu_q_moe_mlp(const void* x, const int32_t* ids, const float* weights, const uint32_t* Wg, const void* sg,
                     const uint32_t* Wu, const void* su, const uint32_t* Wd, const void* sd, const void* residual,
                     int64_t T, int64_t k, int64_t E, int64_t H, int64_t I, int64_t Ho, int type, int out_mode,
                     void* out, void* stream_v) {
  hipStream_t stream = (hipStream_t)stream_v;
  if (!x || !ids || !weights || !out) return SWQ_ERR_NULL;
  int rc = check_codes(Wg, sg);
  if (rc == SWQ_OK) rc = check_codes(Wu, su);
  if (rc == SWQ_OK) rc = check_codes(Wd, sd);
  if (rc != SWQ_OK) return rc;
  if (!type16_ok(type) || (out_mode != type && out_mode != SWQ_LINEAR_F32)) return SWQ_ERR_UNSUPPORTED;
  if (T < 0 || T > kMaxRows || k < 1 || k > SWQ_MAX_CHOSEN || E < 1 || E > SWQ_MAX_EXPERTS) return SWQ_ERR_SHAPE;
  const int64_t P = T * k;
  rc = check_shape(P, H, I);
  if (rc == SWQ_OK) rc = check_shape(P, I, Ho);
  if (rc != SWQ_OK) return rc;
  if (T * H * 2 >= (int64_t(1) << 32) - 16) return SWQ_ERR_SHAPE;   // gathered rows are 32-bit byte offsets
  if (!aligned(x, 16) || !aligned(ids, 4) || !aligned(weights, 4) || !aligned(out, type_bytes(out_mode)) ||
      !aligned(residual, 2))
    return SWQ_ERR_ALIGN;
  if (T == 0) return SWQ_OK;
  const bool f16 = type == SWQ_TYPE_F16;
  MxGemm g{};
  g.x = (const uint16_t*)x;
  g.w = Wg;
  g.s = (const uint8_t*)sg;
  g.w2 = Wu;
  g.s2 = (const uint8_t*)su;
  g.rows = (int)P;
  g.K = (int)H;
  g.N = (int)I;
  g.E = (int)E;
  g.wrows = I;
  g.xsrc = f16 ? kXF16 : kXBf16;
  g.xdiv = (int)k;
  g.type = type;
  g.out_type = SWQ_TYPE_BF16;
  g.hidden_planes = f16;
  g.xrows = (int)T;
  g.vec = 2;
  // The hidden tensor is rounded to x's precision where it leaves the registers: bf16 x to bf16, as the dense
  // MLP's (swiglu_q_mlp), binary16 x to two bf16 planes, 16 bits.  Against the same formulas in 64 bits bf16
  // outputs are off by 0.0019 to 0.0022 of their norm where an unrounded hidden tensor gives 0.0017, the output's own
  // rounding; two planes for bf16 x too would double the down projection's products (4096 tokens, 8 of 64
  // experts, 2048 x 1024: 2 x 153 us in place of 2 x 105, of 517 in all).
  // Few tokens: every slot on its own, no plan, the weighted sum in the down
  // projection.  Else by expert: the workspace holds the plan, the hidden
  // tensor in the plan's order (two planes for binary16), the experts' outputs
  // in the slots' order, and x as planes.
  const bool direct = slot_by_slot(T, k, E, H, I, Ho);
  g.kind = direct ? (int)kFew : mx4_gemm_kind(g);
  const int tile = mx4_gemm_tile(g);
  const int64_t cols = part_columns(P, Ho);
  if (direct) g.ids = ids;
  else g.max_tiles = (int)max_row_tiles(P, E, tile);
  MxGemm d = g;                       // the down projection
  d.w = Wd;
  d.s = (const uint8_t*)sd;
  d.w2 = nullptr;
  d.s2 = nullptr;
  d.K = (int)I;
  d.N = (int)(direct || Ho < cols ? Ho : cols);
  d.wrows = Ho;
  d.xsrc = f16 ? kXPlanes : kXBf16;
  d.out_type = SWQ_TYPE_F32;
  d.hidden_planes = 0;
  d.check_only = 1;
  if (!fits(g) || (direct ? launch_mx4_down(d, weights, (int)k, stream) : launch_mx4_gemm(d, stream)) != hipSuccess)
    return SWQ_ERR_SHAPE;
  d.check_only = 0;
  const PlanLayout l = direct ? PlanLayout{0, 0, 0} : plan_layout(P, E, tile, true);
  const int64_t hidden = align256(P * I * 2) * (f16 ? 2 : 1);
  const int64_t part = l.total + hidden, xplanes = part + (direct ? 0 : align256(P * cols * 4));
  void* ws_v = nullptr;
  rc = stream_workspace(stream, (size_t)(xplanes + (direct ? 0 : planes_bytes(g, T))), &ws_v, kWsSlot);
  if (rc != SWQ_OK) return rc;
  char* ws = (char*)ws_v;
  (void)hipGetLastError();
  if (!direct) {
    const int* perm = nullptr;
    rc = run_plan(g, ws, l, ids, nullptr, tile, stream, &perm);
    if (rc == SWQ_OK) rc = to_planes(g, T, ws + xplanes, stream);
    if (rc != SWQ_OK) return rc;
    g.xperm = perm;
    d.perm = perm;
    d.tiles = g.tiles;
    d.ntiles = g.ntiles;
  }
  g.out = ws + l.total;
  g.out_plane = align256(P * I * 2) / 2;
  rc = check_status(launch_mx4_gemm(g, stream));
  if (rc != SWQ_OK) return rc;
  d.x = (const uint16_t*)(ws + l.total);
  d.plane = g.out_plane;
  if (direct) {
    d.res = (const uint16_t*)residual;
    d.out = out;
    d.out_type = out_mode;
    d.vec = vec_ok(Ho, out, residual, out_mode);
    return check_status(launch_mx4_down(d, weights, (int)k, stream));
  }
  d.out = ws + part;
  for (int64_t n = 0; n < Ho; n += cols) {
    d.N = (int)(Ho - n < cols ? Ho - n : cols);
    d.w = Wd + n * (I / 8);
    d.s = (const uint8_t*)sd + n * (I / 32);
    d.vec = vec_ok(d.N, d.out, nullptr, SWQ_TYPE_F32);
    rc = check_status(launch_mx4_gemm(d, stream));
    if (rc != SWQ_OK) return rc;
    const uint16_t* res = residual ? (const uint16_t*)residual + n : nullptr;
    rc = check_status(launch_combine((const float*)(ws + part), ids, weights, res, T, (int)k, (int)E, d.N, Ho, type,
                                     out_mode, (char*)out + n * type_bytes(out_mode), stream));
    if (rc != SWQ_OK) return rc;
  }
  return SWQ_OK;
}

}  // extern "C"
