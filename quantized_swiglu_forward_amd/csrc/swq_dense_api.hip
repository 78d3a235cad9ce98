// C-ABI entry points of the products with 16-bit weights, the 8-bit activation
// checkpoints, the SwiGLU with checkpoints and the router's loss and gradient (declared in
// include/swiglu_q.h): validation on the host, then launches on the caller's
// stream.
#include <algorithm>

#include "../../include/swiglu_q.h"
#include "swq_dense.h"

using namespace swq;

namespace {

constexpr int kWsSlot = 3;            // this workspace beside the MLP's two and the experts'
constexpr int64_t kMaxRows = int64_t(1) << 30, kMaxK = int64_t(1) << 20;

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }
bool type_ok(int t) { return t == SWQ_TYPE_BF16 || t == SWQ_TYPE_F32 || t == SWQ_TYPE_F16; }
bool type16_ok(int t) { return t == SWQ_TYPE_BF16 || t == SWQ_TYPE_F16; }
bool act_ok(int a) { return a >= SWQ_ACT_NONE && a <= SWQ_ACT_GELU_TANH; }
int64_t align256(int64_t v) { return (v + 255) / 256 * 256; }
int check_status(hipError_t e) { return e == hipSuccess ? SWQ_OK : SWQ_ERR_HIP; }

// Rows, inputs and outputs of a product.
int check_shape(int64_t M, int64_t K, int64_t N) {
  return M < 0 || K <= 0 || N <= 0 || M > kMaxRows || K > kMaxK || N > kMaxK ? SWQ_ERR_SHAPE : SWQ_OK;
}
// Elementwise tensors [R, K].
int check_elements(int64_t R, int64_t K) {
  return R < 0 || K <= 0 || K > kMaxK || R > kMaxRows || R * K >= (int64_t(1) << 41) ? SWQ_ERR_SHAPE : SWQ_OK;
}
// A tensor in 16 bits (2-byte aligned) or a checkpoint (codes of any address).
bool kept_aligned(const void* data, const void* scales) { return scales || aligned(data, 2); }

// `need` bytes of the stream's workspace (none: null).
int take(void* stream, int64_t need, char** ws) {
  if (need == 0) return SWQ_OK;
  void* p = nullptr;
  const int rc = stream_workspace((hipStream_t)stream, (size_t)need, &p, kWsSlot);
  *ws = (char*)p;
  return rc;
}

}  // namespace

extern "C" {

int swiglu_q_dense_linear(const void* x, const void* W, const void* bias, const void* residual, int64_t M, int64_t K,
                          int64_t N, int type, int act, int out_mode, void* out, void* z, void* z_scales,
                          void* stream_v) {
  hipStream_t stream = (hipStream_t)stream_v;
  if (!x || !W || !out || (z_scales && !z)) return SWQ_ERR_NULL;
  if (!type16_ok(type) || !act_ok(act) || (out_mode != type && out_mode != SWQ_LINEAR_F32)) return SWQ_ERR_UNSUPPORTED;
  int rc = check_shape(M, K, N);
  if (rc != SWQ_OK) return rc;
  if (!aligned(x, 16) || !aligned(W, 16) || !aligned(bias, 2) || !aligned(residual, 2) ||
      !aligned(out, type_bytes(out_mode)) || !kept_aligned(z, z_scales))
    return SWQ_ERR_ALIGN;
  if (M == 0) return SWQ_OK;
  DenseGemm g{};
  g.a = (const uint16_t*)x;
  g.b = (const uint16_t*)W;
  g.lda = g.ldb = K;
  g.P = M;
  g.Q = N;
  g.R = K;
  g.type = type;
  g.act = act;
  g.bias = (const uint16_t*)bias;
  g.res = (const uint16_t*)residual;
  g.out = out;
  g.out_type = out_mode;
  g.z = z;
  g.z_scales = (uint8_t*)z_scales;
  if (!plan_dense_gemm(g)) return SWQ_ERR_SHAPE;
  // Workspace: x and W with rows of whole 16-byte units, the partial sums of a split.
  const bool pad = K % 8 != 0 && dense_takes_units(g);
  const int64_t x_bytes = pad ? align256(M * ceil8(K) * 2) : 0, w_bytes = pad ? align256(N * ceil8(K) * 2) : 0;
  char* ws = nullptr;
  rc = take(stream_v, x_bytes + w_bytes + dense_parts_bytes(g), &ws);
  if (rc != SWQ_OK) return rc;
  (void)hipGetLastError();            // before the first launch: an error left by others is not this call's
  if (pad) {
    Prep p{};
    p.rows[0] = {x, nullptr, M, K, (uint16_t*)ws};
    p.rows[1] = {W, nullptr, N, K, (uint16_t*)(ws + x_bytes)};
    rc = check_status(launch_prep(p, type, stream));
    if (rc != SWQ_OK) return rc;
    g.a = p.rows[0].dst;
    g.b = p.rows[1].dst;
    g.lda = g.ldb = ceil8(K);
  }
  g.parts = (float*)(ws + x_bytes + w_bytes);
  return check_status(launch_dense_gemm(g, stream));
}

int swiglu_q_dense_linear_backward(const void* dout, const void* x, const void* x_scales, const void* W, const void* z,
                                   const void* z_scales, int64_t M, int64_t K, int64_t N, int type, int act, void* dx,
                                   void* dW, void* dbias, void* stream_v) {
  hipStream_t stream = (hipStream_t)stream_v;
  if (!dout || (!dx && !dW && !dbias) || (dx && !W) || (dW && !x) || (act != SWQ_ACT_NONE && !z)) return SWQ_ERR_NULL;
  if (!type16_ok(type) || !act_ok(act)) return SWQ_ERR_UNSUPPORTED;
  int rc = check_shape(M, K, N);
  if (rc != SWQ_OK) return rc;
  if (!aligned(dout, 16) || (dx && !aligned(W, 16)) || (dW && !aligned(x, x_scales ? 1 : 16)) || !kept_aligned(z, z_scales) ||
      !aligned(dx, 2) || !aligned(dW, 2) || !aligned(dbias, 2))
    return SWQ_ERR_ALIGN;
  (void)hipGetLastError();
  if (M == 0) {                       // sums of nothing
    hipError_t e = hipSuccess;
    if (dW) e = launch_zero16((uint16_t*)dW, N * K, stream);
    if (dbias && e == hipSuccess) e = launch_zero16((uint16_t*)dbias, N, stream);
    return check_status(e);
  }
  DensePair d{};
  d.x.type = d.x.out_type = d.w.type = d.w.out_type = type;
  d.x.lda = d.w.lda = ceil8(N);
  d.x.ldb = d.w.ldb = ceil8(K);
  d.x.P = M, d.x.Q = K, d.x.R = N;
  d.w.P = N, d.w.Q = K, d.w.R = M;
  d.x.out = dx;
  d.w.out = dW;
  d.N = N;
  if (!plan_dense_pair(d, dx, dW)) return SWQ_ERR_SHAPE;
  // Workspace: dz (where dout itself will not do), x and W with rows of whole 16-byte units, the partial sums of the
  // splits and of the bias's gradient.
  const bool has_dz = (act != SWQ_ACT_NONE || N % 8 != 0) && (dx || dW);
  const bool has_x = dW && (x_scales || K % 8 != 0), has_w = dx && K % 8 != 0;
  const int64_t dz_bytes = has_dz ? align256(M * ceil8(N) * 2) : 0, x_bytes = has_x ? align256(M * ceil8(K) * 2) : 0;
  const int64_t w_bytes = has_w ? align256(N * ceil8(K) * 2) : 0;
  const int64_t x_parts = dx ? align256(dense_parts_bytes(d.x)) : 0, w_parts = dW ? align256(dense_parts_bytes(d.w)) : 0;
  const int64_t n_sums = dbias ? act_parts(M, N) : 0, sums = n_sums > 1 ? n_sums * N * 4 : 0;
  char* ws = nullptr;
  rc = take(stream_v, dz_bytes + x_bytes + w_bytes + x_parts + w_parts + sums, &ws);
  if (rc != SWQ_OK) return rc;
  (void)hipGetLastError();
  char* at = ws;
  const auto next = [&](int64_t bytes) { return (void*)(at += bytes, at - bytes); };
  Prep p{};
  p.dz = has_dz ? (uint16_t*)next(dz_bytes) : nullptr;
  if (has_x) p.rows[0] = {x, (const uint8_t*)x_scales, M, K, (uint16_t*)next(x_bytes)};
  if (has_w) p.rows[1] = {W, nullptr, N, K, (uint16_t*)next(w_bytes)};
  d.x.parts = (float*)next(x_parts);
  d.w.parts = (float*)next(w_parts);
  if (has_dz || dbias) {
    p.dout = (const uint16_t*)dout;
    p.z = Kept{z, (const uint8_t*)z_scales};
    p.M = M;
    p.N = N;
    p.act = act;
    if (n_sums > 1) d.sums = p.sums = (float*)next(sums), d.n_sums = (int)n_sums, d.dbias = (uint16_t*)dbias;
    else p.dbias = (uint16_t*)dbias;
  }
  rc = check_status(launch_prep(p, type, stream));
  if (rc != SWQ_OK || (!dx && !dW && !d.n_sums)) return rc;
  d.x.a = d.w.a = has_dz ? p.dz : (const uint16_t*)dout;
  d.x.b = has_w ? p.rows[1].dst : (const uint16_t*)W;
  d.w.b = has_x ? p.rows[0].dst : (const uint16_t*)x;
  return check_status(launch_dense_pair(d, type, stream));
}

int swiglu_q_mx8_quantize(const void* x, int64_t R, int64_t K, int type, void* codes, void* scales, void* stream) {
  if (!x || !codes || !scales) return SWQ_ERR_NULL;
  if (!type_ok(type)) return SWQ_ERR_UNSUPPORTED;
  const int rc = check_elements(R, K);
  if (rc != SWQ_OK) return rc;
  if (!aligned(x, type_bytes(type))) return SWQ_ERR_ALIGN;
  if (R == 0) return SWQ_OK;
  (void)hipGetLastError();
  return check_status(launch_mx8_quantize(x, R, K, type, codes, (uint8_t*)scales, (hipStream_t)stream));
}

int swiglu_q_mx8_dequantize(const void* codes, const void* scales, int64_t R, int64_t K, int type, void* out,
                            void* stream) {
  if (!codes || !scales || !out) return SWQ_ERR_NULL;
  if (!type_ok(type)) return SWQ_ERR_UNSUPPORTED;
  const int rc = check_elements(R, K);
  if (rc != SWQ_OK) return rc;
  if (!aligned(out, type_bytes(type))) return SWQ_ERR_ALIGN;
  if (R == 0) return SWQ_OK;
  (void)hipGetLastError();
  return check_status(launch_mx8_dequantize(codes, (const uint8_t*)scales, R, K, type, out, (hipStream_t)stream));
}

int swiglu_q_swiglu(const void* gate, const void* up, int64_t R, int64_t K, int type, void* hidden, void* gate_codes,
                    void* gate_scales, void* up_codes, void* up_scales, void* stream) {
  if (!gate || !up || !hidden) return SWQ_ERR_NULL;
  const int kept = !!gate_codes + !!gate_scales + !!up_codes + !!up_scales;
  if (kept != 0 && kept != 4) return SWQ_ERR_NULL;
  if (!type16_ok(type)) return SWQ_ERR_UNSUPPORTED;
  const int rc = check_elements(R, K);
  if (rc != SWQ_OK) return rc;
  if (!aligned(gate, 2) || !aligned(up, 2) || !aligned(hidden, 2)) return SWQ_ERR_ALIGN;
  if (R == 0) return SWQ_OK;
  (void)hipGetLastError();
  return check_status(launch_swiglu((const uint16_t*)gate, (const uint16_t*)up, R, K, type, (uint16_t*)hidden,
                                    gate_codes, (uint8_t*)gate_scales, up_codes, (uint8_t*)up_scales,
                                    (hipStream_t)stream));
}

int swiglu_q_swiglu_backward(const void* dhidden, const void* gate, const void* gate_scales, const void* up,
                             const void* up_scales, int64_t R, int64_t K, int type, void* dgate, void* dup,
                             void* hidden, void* stream) {
  if (!dhidden || !gate || !up || !dgate || !dup) return SWQ_ERR_NULL;
  if (!type16_ok(type)) return SWQ_ERR_UNSUPPORTED;
  const int rc = check_elements(R, K);
  if (rc != SWQ_OK) return rc;
  if (!aligned(dhidden, 2) || !kept_aligned(gate, gate_scales) || !kept_aligned(up, up_scales) || !aligned(dgate, 2) ||
      !aligned(dup, 2) || !aligned(hidden, 2))
    return SWQ_ERR_ALIGN;
  if (R == 0) return SWQ_OK;
  (void)hipGetLastError();
  return check_status(launch_swiglu_backward((const uint16_t*)dhidden, Kept{gate, (const uint8_t*)gate_scales},
                                             Kept{up, (const uint8_t*)up_scales}, R, K, type, (uint16_t*)dgate,
                                             (uint16_t*)dup, (uint16_t*)hidden, (hipStream_t)stream));
}

int swiglu_q_balance_loss(const void* logits, const int32_t* ids, int64_t T, int64_t E, int k, int type, int scoring,
                          float* loss, int32_t* counts, float* slopes, void* stream) {
  if (!logits || !ids || !loss || !counts || !slopes) return SWQ_ERR_NULL;
  if (!type_ok(type) || scoring < SWQ_ROUTE_SOFTMAX || scoring > SWQ_ROUTE_SIGMOID_CHOSEN) return SWQ_ERR_UNSUPPORTED;
  if (T < 0 || T > kMaxRows || E < 1 || E > SWQ_MAX_EXPERTS || k < 1 || k > SWQ_MAX_CHOSEN ||
      T * k >= (int64_t(1) << 31))
    return SWQ_ERR_SHAPE;
  if (!aligned(logits, type_bytes(type)) || !aligned(ids, 4) || !aligned(loss, 4) || !aligned(counts, 4) ||
      !aligned(slopes, 4))
    return SWQ_ERR_ALIGN;
  void* ws = nullptr;
  if (const int64_t need = balance_workspace(T, (int)E)) {
    const int rc = stream_workspace((hipStream_t)stream, (size_t)need, &ws, kWsSlot);
    if (rc != SWQ_OK) return rc;
  }
  (void)hipGetLastError();
  return check_status(
      launch_balance(logits, ids, T, (int)E, k, type, scoring, loss, counts, slopes, ws, (hipStream_t)stream));
}

int swiglu_q_route_backward(const void* logits, const int32_t* ids, const float* dweights, const float* slopes,
                            const float* dloss, int64_t T, int64_t E, int k, int type, int scoring, void* dlogits,
                            void* stream) {
  if (!logits || !ids || !dlogits || (!dweights && !slopes) || (dloss && !slopes)) return SWQ_ERR_NULL;
  if (!type_ok(type) || scoring < SWQ_ROUTE_SOFTMAX || scoring > SWQ_ROUTE_SIGMOID_CHOSEN) return SWQ_ERR_UNSUPPORTED;
  if (T < 0 || T > kMaxRows || E < 1 || E > SWQ_MAX_EXPERTS || k < 1 || k > SWQ_MAX_CHOSEN) return SWQ_ERR_SHAPE;
  if (!aligned(logits, type_bytes(type)) || !aligned(ids, 4) || !aligned(dweights, 4) || !aligned(slopes, 4) ||
      !aligned(dloss, 4) || !aligned(dlogits, type_bytes(type)))
    return SWQ_ERR_ALIGN;
  if (T == 0) return SWQ_OK;
  (void)hipGetLastError();
  return check_status(launch_route_backward(logits, ids, dweights, slopes, dloss, T, (int)E, k, type, scoring, dlogits,
                                            (hipStream_t)stream));
}

}  // extern "C"
