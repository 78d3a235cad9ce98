"""Fused quantized SwiGLU expansion for AMD Instinct MI355X (gfx950).

``hidden = silu(x Wg^T) * (x Wu^T)`` with affine group-quantized Wg/Wu, computed
by the hand-written HIP kernels of ``libswiglu_q.so``.  This module only
marshals arguments into the library's C ABI (``include/swiglu_q.h``): every
step of the computation runs in the HIP kernels, and nothing here falls back
to another implementation.  PyTorch supplies device memory and streams.

Functions with the C names take raw device pointers (ints) or tensors and
return the integer status; ``forward`` / ``debug_gemm_tensors`` are tensor
conveniences that allocate outputs with torch and raise ``SwigluQError``.
"""
from __future__ import annotations

import ctypes
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libswiglu_q.so")

(SWQ_OK, SWQ_ERR_NULL, SWQ_ERR_SHAPE, SWQ_ERR_UNSUPPORTED, SWQ_ERR_ALIGN, SWQ_ERR_HIP, SWQ_ERR_WORKSPACE,
 SWQ_ERR_TOO_LARGE) = range(8)
SWQ_MATCH, SWQ_F32, SWQ_F32_BF16OUT = 0, 1, 2
SWQ_PATH_GEMV, SWQ_PATH_MFMA, SWQ_PATH_AUTO = 0, 1, -1
SWQ_LINEAR_BF16, SWQ_LINEAR_F32, SWQ_LINEAR_F16 = 0, 1, 2
SWQ_TYPE_BF16, SWQ_TYPE_F32, SWQ_TYPE_F16 = 0, 1, 2
SWQ_ROUTE_SOFTMAX, SWQ_ROUTE_SOFTMAX_CHOSEN, SWQ_ROUTE_SIGMOID, SWQ_ROUTE_SIGMOID_CHOSEN = range(4)
SWQ_MAX_EXPERTS, SWQ_MAX_CHOSEN = 1024, 64
SWQ_ACT_NONE, SWQ_ACT_RELU, SWQ_ACT_SILU, SWQ_ACT_GELU, SWQ_ACT_GELU_TANH = range(5)

_lib = None


class SwigluQError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: status {status} ({strerror(status)})" if what else
                         f"status {status} ({strerror(status)})")


def lib():
    """Load ``libswiglu_q.so``; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run `python -m quantized_swiglu_forward_amd.build`")
    _lib = load_library(LIB_PATH)
    return _lib


def load_library(path):
    """A ctypes handle on a build of the library at ``path`` (the product, or
    its LDS-poison debug twin ``libswiglu_q_ldspoison.so``) with every entry
    point's signature declared."""
    L = ctypes.CDLL(path)
    vp, i64, i32, u64 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_uint64
    L.swiglu_q_forward.argtypes = [vp] * 7 + [i64, i64, i64, i32, i32, i32, i32, i32, vp, vp]
    L.swiglu_q_forward.restype = i32
    L.swiglu_q_forward_f16.argtypes = [vp] * 7 + [i64, i64, i64, i32, i32, i32, i32, i32, vp, vp]
    L.swiglu_q_forward_f16.restype = i32
    L.swiglu_q_forward_noalloc.argtypes = [vp] * 7 + [i64, i64, i64, i32, i32, i32, i32, i32, vp, vp]
    L.swiglu_q_forward_noalloc.restype = i32
    L.swiglu_q_linear.argtypes = [vp] * 4 + [i64, i64, i64, i32, i32, i32, vp, vp]
    L.swiglu_q_linear.restype = i32
    L.swiglu_q_mlp.argtypes = [vp] * 11 + [i64, i64, i64, i64, i32, i32, i32, i32, i32, i32, i32, vp, vp]
    L.swiglu_q_mlp.restype = i32
    L.swiglu_q_debug_gemm.argtypes = [vp] * 7 + [i64, i64, i64, i32, i32, i32, i32, i32, vp, vp, vp]
    L.swiglu_q_debug_gemm.restype = i32
    L.swiglu_q_mx4_quantize.argtypes = [vp, i64, i64, i32, vp, vp, vp]
    L.swiglu_q_mx4_quantize.restype = i32
    L.swiglu_q_mx4_dequantize.argtypes = [vp, vp, i64, i64, i32, vp, vp]
    L.swiglu_q_mx4_dequantize.restype = i32
    L.swiglu_q_mx4_linear.argtypes = [vp] * 4 + [i64, i64, i64, i32, i32, vp, vp]
    L.swiglu_q_mx4_linear.restype = i32
    L.swiglu_q_mx4_matmul.argtypes = [vp] * 4 + [i64, i64, i64, i32, vp, vp]
    L.swiglu_q_mx4_matmul.restype = i32
    L.swiglu_q_mx4_grouped_linear.argtypes = [vp] * 4 + [i64, i64, i64, i64, i32, i32, vp, vp]
    L.swiglu_q_mx4_grouped_linear.restype = i32
    L.swiglu_q_route.argtypes = [vp, i64, i64, i32, i32, i32, vp, vp, vp]
    L.swiglu_q_route.restype = i32
    L.swiglu_q_moe_mlp.argtypes = [vp] * 10 + [i64] * 6 + [i32, i32, vp, vp]
    L.swiglu_q_moe_mlp.restype = i32
    L.swiglu_q_mx8_quantize.argtypes = [vp, i64, i64, i32, vp, vp, vp]
    L.swiglu_q_mx8_quantize.restype = i32
    L.swiglu_q_mx8_dequantize.argtypes = [vp, vp, i64, i64, i32, vp, vp]
    L.swiglu_q_mx8_dequantize.restype = i32
    L.swiglu_q_dense_linear.argtypes = [vp] * 4 + [i64, i64, i64, i32, i32, i32, vp, vp, vp, vp]
    L.swiglu_q_dense_linear.restype = i32
    L.swiglu_q_dense_linear_backward.argtypes = [vp] * 6 + [i64, i64, i64, i32, i32, vp, vp, vp, vp]
    L.swiglu_q_dense_linear_backward.restype = i32
    L.swiglu_q_swiglu.argtypes = [vp, vp, i64, i64, i32] + [vp] * 6
    L.swiglu_q_swiglu.restype = i32
    L.swiglu_q_swiglu_backward.argtypes = [vp] * 5 + [i64, i64, i32] + [vp] * 4
    L.swiglu_q_swiglu_backward.restype = i32
    L.swiglu_q_balance_loss.argtypes = [vp, vp, i64, i64, i32, i32, i32, vp, vp, vp, vp]
    L.swiglu_q_balance_loss.restype = i32
    L.swiglu_q_route_backward.argtypes = [vp] * 5 + [i64, i64, i32, i32, i32, vp, vp]
    L.swiglu_q_route_backward.restype = i32
    L.swiglu_q_supported.argtypes = [i64, i32, i32, i32, i32, i32]
    L.swiglu_q_supported.restype = i32
    L.swiglu_q_set_m_threshold.argtypes = [i32]
    L.swiglu_q_set_m_threshold.restype = None
    L.swiglu_q_path_for.argtypes = [i64, i64, i64]
    L.swiglu_q_path_for.restype = i32
    L.swiglu_q_get_m_threshold.argtypes = []
    L.swiglu_q_get_m_threshold.restype = i32
    L.swiglu_q_call_count.argtypes = [i32]
    L.swiglu_q_call_count.restype = u64
    L.swiglu_q_reset_counts.argtypes = []
    L.swiglu_q_reset_counts.restype = None
    L.swiglu_q_staging_bytes.argtypes = [i64, i64, i64, i32, i32, i32, i32, i32]
    L.swiglu_q_staging_bytes.restype = i64
    L.swiglu_q_set_max_calls.argtypes = [i64]
    L.swiglu_q_set_max_calls.restype = None
    L.swiglu_q_under_cap.argtypes = []
    L.swiglu_q_under_cap.restype = i32
    L.swiglu_q_strerror.argtypes = [i32]
    L.swiglu_q_strerror.restype = ctypes.c_char_p
    L.swiglu_q_workspace_bytes.argtypes = [i64, i64, i64, i32, i32, i32, i32]
    L.swiglu_q_workspace_bytes.restype = i64
    L.swiglu_q_release_workspace.argtypes = []
    L.swiglu_q_release_workspace.restype = i32
    L.swiglu_q_version.argtypes = []
    L.swiglu_q_version.restype = ctypes.c_char_p
    return L


def _ptr(a):
    if a is None:
        return None
    if isinstance(a, int):
        return a
    return a.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


# ---- the C entry points, same names ---------------------------------------

def swiglu_q_forward(x, Wg, sg, bg, Wu, su, bu, M, H, I, bits_g, gs_g, bits_u, gs_u,
                     precision_mode, out, stream=None) -> int:
    return lib().swiglu_q_forward(_ptr(x), _ptr(Wg), _ptr(sg), _ptr(bg), _ptr(Wu), _ptr(su), _ptr(bu),
                                  M, H, I, bits_g, gs_g, bits_u, gs_u, precision_mode, _ptr(out),
                                  _stream(stream))


def swiglu_q_forward_f16(x, Wg, sg, bg, Wu, su, bu, M, H, I, bits_g, gs_g, bits_u, gs_u,
                         precision_mode, out, stream=None) -> int:
    return lib().swiglu_q_forward_f16(_ptr(x), _ptr(Wg), _ptr(sg), _ptr(bg), _ptr(Wu), _ptr(su), _ptr(bu),
                                      M, H, I, bits_g, gs_g, bits_u, gs_u, precision_mode, _ptr(out),
                                      _stream(stream))


def swiglu_q_forward_noalloc(x, Wg, sg, bg, Wu, su, bu, M, H, I, bits_g, gs_g, bits_u, gs_u,
                             precision_mode, out, stream=None) -> int:
    return lib().swiglu_q_forward_noalloc(_ptr(x), _ptr(Wg), _ptr(sg), _ptr(bg), _ptr(Wu), _ptr(su), _ptr(bu),
                                          M, H, I, bits_g, gs_g, bits_u, gs_u, precision_mode, _ptr(out),
                                          _stream(stream))


def swiglu_q_linear(x, W, s, b, M, K, N, bits, gs, out_mode, out, stream=None) -> int:
    return lib().swiglu_q_linear(_ptr(x), _ptr(W), _ptr(s), _ptr(b), M, K, N, bits, gs, out_mode, _ptr(out),
                                 _stream(stream))


def swiglu_q_mlp(x, Wg, sg, bg, Wu, su, bu, Wd, sd, bd, residual, M, H, I, Ho, bits_g, gs_g, bits_u, gs_u,
                 bits_d, gs_d, out_mode, out, stream=None) -> int:
    return lib().swiglu_q_mlp(_ptr(x), _ptr(Wg), _ptr(sg), _ptr(bg), _ptr(Wu), _ptr(su), _ptr(bu), _ptr(Wd),
                              _ptr(sd), _ptr(bd), _ptr(residual), M, H, I, Ho, bits_g, gs_g, bits_u, gs_u, bits_d,
                              gs_d, out_mode, _ptr(out), _stream(stream))


def swiglu_q_mx4_quantize(x, R, K, type, codes, scales, stream=None) -> int:
    return lib().swiglu_q_mx4_quantize(_ptr(x), R, K, type, _ptr(codes), _ptr(scales), _stream(stream))


def swiglu_q_mx4_dequantize(codes, scales, R, K, type, out, stream=None) -> int:
    return lib().swiglu_q_mx4_dequantize(_ptr(codes), _ptr(scales), R, K, type, _ptr(out), _stream(stream))


def swiglu_q_mx4_linear(x, W, s, residual, M, K, N, type, out_mode, out, stream=None) -> int:
    return lib().swiglu_q_mx4_linear(_ptr(x), _ptr(W), _ptr(s), _ptr(residual), M, K, N, type, out_mode, _ptr(out),
                                     _stream(stream))


def swiglu_q_mx4_matmul(A, sa, W, sw, M, K, N, out_mode, out, stream=None) -> int:
    return lib().swiglu_q_mx4_matmul(_ptr(A), _ptr(sa), _ptr(W), _ptr(sw), M, K, N, out_mode, _ptr(out),
                                     _stream(stream))


def swiglu_q_mx4_grouped_linear(x, offsets, W, s, P, E, K, N, type, out_mode, out, stream=None) -> int:
    return lib().swiglu_q_mx4_grouped_linear(_ptr(x), _ptr(offsets), _ptr(W), _ptr(s), P, E, K, N, type, out_mode,
                                             _ptr(out), _stream(stream))


def swiglu_q_route(logits, T, E, k, type, scoring, ids, weights, stream=None) -> int:
    return lib().swiglu_q_route(_ptr(logits), T, E, k, type, scoring, _ptr(ids), _ptr(weights), _stream(stream))


def swiglu_q_moe_mlp(x, ids, weights, Wg, sg, Wu, su, Wd, sd, residual, T, k, E, H, I, Ho, type, out_mode, out,
                     stream=None) -> int:
    return lib().swiglu_q_moe_mlp(_ptr(x), _ptr(ids), _ptr(weights), _ptr(Wg), _ptr(sg), _ptr(Wu), _ptr(su), _ptr(Wd),
                                  _ptr(sd), _ptr(residual), T, k, E, H, I, Ho, type, out_mode, _ptr(out),
                                  _stream(stream))


def swiglu_q_mx8_quantize(x, R, K, type, codes, scales, stream=None) -> int:
    return lib().swiglu_q_mx8_quantize(_ptr(x), R, K, type, _ptr(codes), _ptr(scales), _stream(stream))


def swiglu_q_mx8_dequantize(codes, scales, R, K, type, out, stream=None) -> int:
    return lib().swiglu_q_mx8_dequantize(_ptr(codes), _ptr(scales), R, K, type, _ptr(out), _stream(stream))


def swiglu_q_dense_linear(x, W, bias, residual, M, K, N, type, act, out_mode, out, z=None, z_scales=None,
                          stream=None) -> int:
    return lib().swiglu_q_dense_linear(_ptr(x), _ptr(W), _ptr(bias), _ptr(residual), M, K, N, type, act, out_mode,
                                       _ptr(out), _ptr(z), _ptr(z_scales), _stream(stream))


def swiglu_q_dense_linear_backward(dout, x, x_scales, W, z, z_scales, M, K, N, type, act, dx, dW, dbias,
                                   stream=None) -> int:
    return lib().swiglu_q_dense_linear_backward(_ptr(dout), _ptr(x), _ptr(x_scales), _ptr(W), _ptr(z), _ptr(z_scales),
                                                M, K, N, type, act, _ptr(dx), _ptr(dW), _ptr(dbias), _stream(stream))


def swiglu_q_swiglu(gate, up, R, K, type, hidden, gate_codes=None, gate_scales=None, up_codes=None, up_scales=None,
                    stream=None) -> int:
    return lib().swiglu_q_swiglu(_ptr(gate), _ptr(up), R, K, type, _ptr(hidden), _ptr(gate_codes), _ptr(gate_scales),
                                 _ptr(up_codes), _ptr(up_scales), _stream(stream))


def swiglu_q_swiglu_backward(dhidden, gate, gate_scales, up, up_scales, R, K, type, dgate, dup, hidden=None,
                             stream=None) -> int:
    return lib().swiglu_q_swiglu_backward(_ptr(dhidden), _ptr(gate), _ptr(gate_scales), _ptr(up), _ptr(up_scales), R, K,
                                          type, _ptr(dgate), _ptr(dup), _ptr(hidden), _stream(stream))


def swiglu_q_balance_loss(logits, ids, T, E, k, type, scoring, loss, counts, slopes, stream=None) -> int:
    return lib().swiglu_q_balance_loss(_ptr(logits), _ptr(ids), T, E, k, type, scoring, _ptr(loss), _ptr(counts),
                                       _ptr(slopes), _stream(stream))


def swiglu_q_route_backward(logits, ids, dweights, slopes, dloss, T, E, k, type, scoring, dlogits, stream=None) -> int:
    return lib().swiglu_q_route_backward(_ptr(logits), _ptr(ids), _ptr(dweights), _ptr(slopes), _ptr(dloss), T, E, k,
                                         type, scoring, _ptr(dlogits), _stream(stream))


def swiglu_q_path_for(M, H, I) -> int:
    return lib().swiglu_q_path_for(M, H, I)


def swiglu_q_debug_gemm(x, Wg, sg, bg, Wu, su, bu, M, H, I, bits_g, gs_g, bits_u, gs_u, path,
                        gate_out, up_out, stream=None) -> int:
    return lib().swiglu_q_debug_gemm(_ptr(x), _ptr(Wg), _ptr(sg), _ptr(bg), _ptr(Wu), _ptr(su), _ptr(bu),
                                     M, H, I, bits_g, gs_g, bits_u, gs_u, path, _ptr(gate_out),
                                     _ptr(up_out), _stream(stream))


def swiglu_q_supported(H, bits_g, gs_g, bits_u, gs_u, precision_mode) -> int:
    return lib().swiglu_q_supported(H, bits_g, gs_g, bits_u, gs_u, precision_mode)


def swiglu_q_set_m_threshold(T: int) -> None:
    lib().swiglu_q_set_m_threshold(T)


def swiglu_q_get_m_threshold() -> int:
    return lib().swiglu_q_get_m_threshold()


def swiglu_q_call_count(path: int) -> int:
    return lib().swiglu_q_call_count(path)


def swiglu_q_reset_counts() -> None:
    lib().swiglu_q_reset_counts()


def swiglu_q_set_max_calls(n: int) -> None:
    lib().swiglu_q_set_max_calls(n)


def swiglu_q_under_cap() -> int:
    return lib().swiglu_q_under_cap()


def swiglu_q_strerror(status: int) -> str:
    return lib().swiglu_q_strerror(status).decode()


def swiglu_q_workspace_bytes(M, H, I, bits_g, gs_g, bits_u, gs_u) -> int:
    return lib().swiglu_q_workspace_bytes(M, H, I, bits_g, gs_g, bits_u, gs_u)


def swiglu_q_staging_bytes(M, H, I, bits_g, gs_g, bits_u, gs_u, path=SWQ_PATH_AUTO) -> int:
    return lib().swiglu_q_staging_bytes(M, H, I, bits_g, gs_g, bits_u, gs_u, path)


def swiglu_q_release_workspace() -> int:
    return lib().swiglu_q_release_workspace()


def swiglu_q_version() -> str:
    return lib().swiglu_q_version().decode()


strerror = swiglu_q_strerror


# ---- tensor conveniences ----------------------------------------------------
#
# Like the pages' host entry, these take activations of any leading shape
# [..., H]: the leading dimensions are collapsed into M rows (which must then be
# one contiguous [M, H] block) and restored on the output ("mlx-bun 0.0.7 ->
# 0.0.9" diff, page 42, fused-swiglu-kernel.ts, host entry).

_BITS16 = ("torch.bfloat16", "torch.int16", "torch.uint16")


def _rows(x, what, f16=False):
    """(x as [M, H], leading shape) for bf16 activations (or their int16/uint16
    bit patterns; with f16, float16 activations); raises for any other dtype
    or a non-contiguous tensor."""
    ok = _BITS16 + (("torch.float16",) if f16 else ())
    if str(x.dtype) not in ok:
        raise TypeError(f"{what}: x must be bfloat16{' or float16' if f16 else ''} "
                        f"(or its 16-bit patterns), not {x.dtype}")
    if x.dim() < 1:
        raise ValueError(f"{what}: x needs at least one dimension")
    if not x.is_contiguous():
        raise ValueError(f"{what}: x must be contiguous (rows are read without strides)")
    lead = tuple(x.shape[:-1])
    return x.reshape(-1, x.shape[-1]), lead


def forward(x, wg, sg, bg, wu, su, bu, bits_g, gs_g, bits_u=None, gs_u=None,
            mode=SWQ_MATCH, out=None, stream=None):
    """``hidden`` for device tensors: x [..., H] (bf16 or int16/uint16 bit
    patterns), packed codes int32/uint32 [I, H*bits/32], scales/biases bf16
    [I, H/gs].  float16 x (with float16 scales and biases) runs
    swiglu_q_forward_f16.  Returns ``out`` ([..., I]: float32 in SWQ_F32,
    else x's 16-bit type)."""
    import torch
    bits_u = bits_g if bits_u is None else bits_u
    gs_u = gs_g if gs_u is None else gs_u
    x2, lead = _rows(x, "forward", f16=True)
    f16 = x.dtype == torch.float16
    if any((t.dtype == torch.float16) != f16 for t in (sg, bg, su, bu)):
        raise TypeError("forward: scales and biases must have x's type (float16 with float16 x, bf16 otherwise)")
    M, H = int(x2.shape[0]), int(x2.shape[1])
    I = int(wg.shape[0])
    if out is None:
        dt = torch.float32 if mode == SWQ_F32 else (torch.float16 if f16 else torch.bfloat16)
        out = torch.empty(lead + (I,), dtype=dt, device=x.device)
    entry = swiglu_q_forward_f16 if f16 else swiglu_q_forward
    rc = entry(x2, wg, sg, bg, wu, su, bu, M, H, I, bits_g, gs_g, bits_u, gs_u, mode, out, stream)
    if rc != SWQ_OK:
        raise SwigluQError(rc, entry.__name__)
    return out


def linear(x, w, s, b, bits, gs, out_mode=SWQ_LINEAR_BF16, out=None, stream=None):
    """``x W^T`` for device tensors: x [..., K] bf16, packed codes [N, K*bits/32],
    scales/biases bf16 [N, K/gs].  Returns ``out`` ([..., N], bf16 or float32)."""
    import torch
    x2, lead = _rows(x, "linear")
    M, K = int(x2.shape[0]), int(x2.shape[1])
    N = int(w.shape[0])
    if out is None:
        dt = torch.float32 if out_mode == SWQ_LINEAR_F32 else torch.bfloat16
        out = torch.empty(lead + (N,), dtype=dt, device=x.device)
    rc = swiglu_q_linear(x2, w, s, b, M, K, N, bits, gs, out_mode, out, stream)
    if rc != SWQ_OK:
        raise SwigluQError(rc, "swiglu_q_linear")
    return out


def mlp(x, wg, sg, bg, wu, su, bu, wd, sd, bd, spec_g, spec_u, spec_d, residual=None,
        out_mode=SWQ_LINEAR_BF16, out=None, stream=None):
    """``residual + (silu(x Wg^T) * (x Wu^T)) Wd^T`` for device tensors; each
    spec is (bits, group size); Wd is [Ho, I*bits_d/32]; x is [..., H] and the
    residual, when given, bf16 [..., Ho].  Returns ``out`` ([..., Ho], bf16 or
    float32 by out_mode)."""
    import torch
    x2, lead = _rows(x, "mlp")
    M, H = int(x2.shape[0]), int(x2.shape[1])
    I, Ho = int(wg.shape[0]), int(wd.shape[0])
    if residual is not None:
        residual, rlead = _rows(residual, "mlp residual")
        if rlead != lead or int(residual.shape[1]) != Ho:
            raise ValueError(f"mlp: residual must be [..., {Ho}] with x's leading shape {lead}")
    if out is None:
        dt = torch.float32 if out_mode == SWQ_LINEAR_F32 else torch.bfloat16
        out = torch.empty(lead + (Ho,), dtype=dt, device=x.device)
    rc = swiglu_q_mlp(x2, wg, sg, bg, wu, su, bu, wd, sd, bd, residual, M, H, I, Ho, spec_g[0], spec_g[1],
                      spec_u[0], spec_u[1], spec_d[0], spec_d[1], out_mode, out, stream)
    if rc != SWQ_OK:
        raise SwigluQError(rc, "swiglu_q_mlp")
    return out


# ---- microscaled 4-bit floating point (MXFP4), the router, the experts' MLP ----
#
# Codes are int32 (or uint32) words [..., K/8], scales uint8 [..., K/32];
# experts are a leading dimension.  Every tensor must be contiguous and on x's
# GPU; types and shapes that the library does not take raise here.  A call
# goes to the current stream of x's GPU unless it is given one.  Small calls
# cost as much here as on the GPU, so the checks are kept short.

_types = {}      # torch type -> SWQ_TYPE_*; the rest is set with it
_dtypes = ()     # SWQ_TYPE_* -> torch type
_words = ()      # types of codes
_bytes = _int8 = _int32 = _float32 = None
_raw_stream = _device_now = _on_device = None   # torch's current stream of a GPU, current GPU, GPU guard
# torch's allocation by shape and strides on the current GPU, without its dispatcher (so no mode that watches or fills new
# tensors sees it; the kernels write every element); its public one where this torch has no such call
_fresh = None


def _load_types():
    global _types, _dtypes, _words, _bytes, _int8, _int32, _float32, _raw_stream, _device_now, _on_device, _fresh
    import torch
    _dtypes = (torch.bfloat16, torch.float32, torch.float16)
    _words = (torch.int32, torch.uint32)
    _bytes, _int8, _int32, _float32 = torch.uint8, torch.int8, torch.int32, torch.float32
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda dev: torch.cuda.current_stream(dev).cuda_stream)
    _device_now = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    _on_device = torch.cuda.device
    guards = getattr(getattr(torch._C, "_dynamo", None), "guards", None)
    _fresh = getattr(guards, "_empty_strided_cuda", None) or (
        lambda shape, stride, dtype: torch.empty_strided(shape, stride, dtype=dtype, device="cuda"))
    _types = {t: i for i, t in enumerate(_dtypes)}
    return _types


def _type(t, what, wide=True):
    code = (_types or _load_types()).get(t.dtype, -1)
    if code < 0 or (code == SWQ_TYPE_F32 and not wide):
        raise TypeError(f"{what}: {t.dtype} is not a supported type")
    return code


def _same_place(what, x, *tensors):
    """x's GPU; raises for a tensor that is elsewhere or not contiguous."""
    dev = x.get_device()
    if dev < 0:
        raise ValueError(f"{what}: every tensor must be on one GPU")
    if not x.is_contiguous():
        raise ValueError(f"{what}: every tensor must be contiguous")
    for t in tensors:
        if t is not None:
            if t.get_device() != dev:
                raise ValueError(f"{what}: every tensor must be on one GPU")
            if not t.is_contiguous():
                raise ValueError(f"{what}: every tensor must be contiguous")
    return dev


def _mx4_shape(codes, scales, what, K=-1, dims=2):
    """The leading sizes of a matrix of codes and scales."""
    _types or _load_types()
    if codes.dtype not in _words or scales.dtype is not _bytes:
        raise TypeError(f"{what}: codes must be int32 or uint32 words and scales uint8")
    c, s = codes.shape, scales.shape
    if len(c) != dims or len(s) != dims or c[-1] != 4 * s[-1] or c[:-1] != s[:-1]:
        raise ValueError(f"{what}: codes {tuple(c)} and scales {tuple(s)} are not one "
                         f"{dims}-dimensional MXFP4 matrix")
    if K >= 0 and c[-1] * 8 != K:
        raise ValueError(f"{what}: the weights have {c[-1] * 8} inputs, x has {K}")
    if K == 0:                                # (so that the callers' test for no rows is x.numel() == 0)
        raise ValueError(f"{what}: a product needs inputs (K = 0)")
    return c[:-1]


def _new(shape, dtype, x, dev):
    """An uninitialised tensor on x's GPU dev (new_empty takes half as long again)."""
    if dev != _device_now():
        return x.new_empty(shape, dtype=dtype)
    if len(shape) == 2:                      # (tuples, as it insists on)
        r, c = shape
        return _fresh((r, c), (c or 1, 1), dtype)
    return _fresh(*_laid_out(shape), dtype)


def _several(shape, dtypes, x, dev):
    """Uninitialised tensors of one shape on x's GPU dev (a third of a microsecond each sooner than one by one)."""
    if dev != _device_now():
        return [x.new_empty(shape, dtype=t) for t in dtypes]
    shape, stride = _laid_out(shape)
    return [_fresh(shape, stride, t) for t in dtypes]


def _laid_out(shape):
    """The shape and the strides of a contiguous tensor, as tuples."""
    if len(shape) == 2:
        r, c = shape
        return (r, c), (c or 1, 1)
    stride, step = [], 1
    for k in reversed(shape):
        stride.append(step)
        step *= k or 1
    return tuple(shape), tuple(stride[::-1])


def _out(out, shape, dtype, x, what):
    if out is None:
        return x.new_empty(shape, dtype=dtype)
    if out.dtype != dtype or out.shape != tuple(shape) or not out.is_contiguous() \
            or out.get_device() != x.get_device():
        raise ValueError(f"{what}: out must be a contiguous {dtype} tensor of shape {tuple(shape)} on x's GPU")
    return out


def _out_mode(mode, t, what):
    if mode is None:
        return t
    if mode != t and mode != SWQ_LINEAR_F32:
        raise ValueError(f"{what}: out_mode must be x's type or SWQ_LINEAR_F32")
    return mode


def _residual(residual, x, shape, what):
    if residual is None:
        return None
    if residual.dtype != x.dtype or residual.shape != tuple(shape):
        raise ValueError(f"{what}: residual must be {x.dtype} of shape {tuple(shape)}")
    return residual.data_ptr()


def _call(fn, dev, stream, *args):
    """The entry point on the stream (by default the current one) of GPU dev."""
    if stream is None:
        stream = _raw_stream(dev)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    if dev == _device_now():
        rc = fn(*args, stream)
    else:
        with _on_device(dev):
            rc = fn(*args, stream)
    if rc != SWQ_OK:
        raise SwigluQError(rc, fn.__name__)


def mx4_quantize(x, codes=None, scales=None, stream=None):
    """(codes int32 [..., K/8], scales uint8 [..., K/32]) of x [..., K] (bf16,
    float16 or float32; K a multiple of 32)."""
    t = _type(x, "mx4_quantize")
    shape = x.shape
    if len(shape) < 1 or shape[-1] % 32 or shape[-1] == 0:
        raise ValueError("mx4_quantize: the last dimension must be a positive multiple of 32")
    dev = _same_place("mx4_quantize", x)
    K, n, lead = shape[-1], x.numel(), shape[:-1]
    codes = (x.new_empty(lead + (K // 8,), dtype=_int32) if codes is None
             else _out(codes, lead + (K // 8,), _int32, x, "mx4_quantize codes"))
    scales = (x.new_empty(lead + (K // 32,), dtype=_bytes) if scales is None
              else _out(scales, lead + (K // 32,), _bytes, x, "mx4_quantize scales"))
    if n:
        _call((_lib or lib()).swiglu_q_mx4_quantize, dev, stream, x.data_ptr(), n // K, K, t, codes.data_ptr(),
              scales.data_ptr())
    return codes, scales


def mx4_dequantize(codes, scales, dtype=None, out=None, stream=None):
    """The values [..., K] of codes and scales, in bf16 (default), float16 or float32."""
    lead = _mx4_shape(codes, scales, "mx4_dequantize", dims=codes.dim())
    dtype = _dtypes[0] if dtype is None else dtype
    dev = _same_place("mx4_dequantize", codes, scales)
    K = codes.shape[-1] * 8
    shape = lead + (K,)
    out = codes.new_empty(shape, dtype=dtype) if out is None else _out(out, shape, dtype, codes, "mx4_dequantize")
    t, n = _type(out, "mx4_dequantize"), out.numel()
    if n:
        _call((_lib or lib()).swiglu_q_mx4_dequantize, dev, stream, codes.data_ptr(), scales.data_ptr(), n // K, K, t,
              out.data_ptr())
    return out


def mx4_linear(x, w, s, residual=None, out_mode=None, out=None, stream=None):
    """``x W^T`` (+ residual) with MXFP4 W [N, K]: x [..., K] bf16 or float16.
    Returns ``out`` [..., N] in x's type, or float32 with SWQ_LINEAR_F32."""
    t = _type(x, "mx4_linear", wide=False)
    K = x.shape[-1]
    N, = _mx4_shape(w, s, "mx4_linear", K)
    mode = _out_mode(out_mode, t, "mx4_linear")
    shape = x.shape[:-1] + (N,)
    res = _residual(residual, x, shape, "mx4_linear")
    dev = _same_place("mx4_linear", x, w, s, residual)
    out = x.new_empty(shape, dtype=_dtypes[mode]) if out is None else _out(out, shape, _dtypes[mode], x, "mx4_linear")
    n = x.numel()
    if n and N:
        _call((_lib or lib()).swiglu_q_mx4_linear, dev, stream, x.data_ptr(), w.data_ptr(), s.data_ptr(), res, n // K,
              K, N, t, mode, out.data_ptr())
    return out


def mx4_matmul(a, sa, w, sw, out_mode=SWQ_LINEAR_BF16, out=None, stream=None):
    """``A W^T`` of two MXFP4 matrices: A [..., K], W [N, K].  Returns ``out``
    [..., N] (SWQ_LINEAR_BF16, _F32 or _F16)."""
    lead = _mx4_shape(a, sa, "mx4_matmul", dims=a.dim())
    K = a.shape[-1] * 8
    N, = _mx4_shape(w, sw, "mx4_matmul", K)
    if out_mode not in (SWQ_LINEAR_BF16, SWQ_LINEAR_F32, SWQ_LINEAR_F16):
        raise ValueError("mx4_matmul: unknown out_mode")
    dev = _same_place("mx4_matmul", a, sa, w, sw)
    shape, dtype = lead + (N,), _dtypes[out_mode]
    out = a.new_empty(shape, dtype=dtype) if out is None else _out(out, shape, dtype, a, "mx4_matmul")
    n = a.numel()
    if n and N:
        _call((_lib or lib()).swiglu_q_mx4_matmul, dev, stream, a.data_ptr(), sa.data_ptr(), w.data_ptr(),
              sw.data_ptr(), n * 8 // K, K, N, out_mode, out.data_ptr())
    return out


def mx4_grouped_linear(x, offsets, w, s, out_mode=None, out=None, stream=None):
    """``x[p] W[e]^T`` for rows sorted by expert: x [P, K] bf16 or float16, offsets
    int32 [E + 1] on the device (expert e has rows offsets[e] .. offsets[e+1]),
    W [E, N, K].  Returns ``out`` [P, N]; rows of no expert are zero."""
    t = _type(x, "mx4_grouped_linear", wide=False)
    if x.dim() != 2:
        raise ValueError("mx4_grouped_linear: x must be [rows, K]")
    P, K = x.shape
    E, N = _mx4_shape(w, s, "mx4_grouped_linear", K, dims=3)
    if offsets.dtype != _int32 or offsets.shape != (E + 1,):
        raise ValueError(f"mx4_grouped_linear: offsets must be int32 [{E + 1}]")
    mode = _out_mode(out_mode, t, "mx4_grouped_linear")
    dev = _same_place("mx4_grouped_linear", x, offsets, w, s)
    dtype = _dtypes[mode]
    out = x.new_empty((P, N), dtype=dtype) if out is None else _out(out, (P, N), dtype, x, "mx4_grouped_linear")
    if P and N:
        _call((_lib or lib()).swiglu_q_mx4_grouped_linear, dev, stream, x.data_ptr(), offsets.data_ptr(), w.data_ptr(),
              s.data_ptr(), P, E, K, N, t, mode, out.data_ptr())
    return out


def route(logits, k, scoring=SWQ_ROUTE_SOFTMAX, ids=None, weights=None, stream=None):
    """(ids int32 [..., k], weights float32 [..., k]): the k largest of each row
    of logits [..., E] and their routing weights (SWQ_ROUTE_*); -1 and 0 where
    fewer than k logits are above -inf."""
    t = _type(logits, "route")
    shape = logits.shape
    if len(shape) < 1:
        raise ValueError("route: logits need at least one dimension")
    dev = _same_place("route", logits)
    E, lead, n = shape[-1], shape[:-1], logits.numel()
    each = lead + (k,)
    ids = logits.new_empty(each, dtype=_int32) if ids is None else _out(ids, each, _int32, logits, "route ids")
    weights = (logits.new_empty(each, dtype=_float32) if weights is None
               else _out(weights, each, _float32, logits, "route weights"))
    if ids.numel() or n:
        _call((_lib or lib()).swiglu_q_route, dev, stream, logits.data_ptr(), n // max(E, 1), E, k, t, scoring,
              ids.data_ptr(), weights.data_ptr())
    return ids, weights


def moe_mlp(x, ids, weights, wg, sg, wu, su, wd, sd, residual=None, out_mode=None, out=None, stream=None):
    """``residual + sum_j weights[t, j] MLP_e(x[t])``, e = ids[t, j], the MLP of
    each expert being ``(silu(x Wg^T) * (x Wu^T)) Wd^T`` with MXFP4 weights
    Wg, Wu [E, I, H], Wd [E, Ho, I].  x [..., H] bf16 or float16, ids int32 and
    weights float32 [..., k] (``route``'s output; an id outside the experts is
    skipped).  Returns ``out`` [..., Ho] in x's type, or float32 with
    SWQ_LINEAR_F32."""
    t = _type(x, "moe_mlp", wide=False)
    H, lead = x.shape[-1], x.shape[:-1]
    E, I = _mx4_shape(wg, sg, "moe_mlp gate", H, dims=3)
    if _mx4_shape(wu, su, "moe_mlp up", H, dims=3) != (E, I):
        raise ValueError("moe_mlp: gate and up differ in shape")
    Ed, Ho = _mx4_shape(wd, sd, "moe_mlp down", I, dims=3)
    if Ed != E:
        raise ValueError(f"moe_mlp: {E} experts in the gate, {Ed} in the down projection")
    if ids.dtype != _int32 or weights.dtype != _float32 or ids.shape != weights.shape \
            or ids.dim() < 1 or ids.shape[:-1] != lead:
        raise ValueError(f"moe_mlp: ids must be int32 and weights float32 of shape {tuple(lead) + ('k',)}")
    mode = _out_mode(out_mode, t, "moe_mlp")
    shape = lead + (Ho,)
    res = _residual(residual, x, shape, "moe_mlp")
    dev = _same_place("moe_mlp", x, ids, weights, wg, sg, wu, su, wd, sd, residual)
    out = x.new_empty(shape, dtype=_dtypes[mode]) if out is None else _out(out, shape, _dtypes[mode], x, "moe_mlp")
    n = x.numel()
    if n and Ho:
        _call((_lib or lib()).swiglu_q_moe_mlp, dev, stream, x.data_ptr(), ids.data_ptr(), weights.data_ptr(),
              wg.data_ptr(), sg.data_ptr(), wu.data_ptr(), su.data_ptr(), wd.data_ptr(), sd.data_ptr(), res, n // H,
              ids.shape[-1], E, H, I, Ho, t, mode, out.data_ptr())
    return out


# ---- products with 16-bit weights, and training ---------------------------------
#
# Rules as above.  A checkpoint is a pair (codes int8 [..., K], scales uint8
# [..., ceil(K / 32)]), as mx8_quantize returns it.

def _mx8(kept, what):
    """The codes and scales of a checkpoint."""
    _types or _load_types()
    codes, scales = kept
    if codes.dtype is not _int8 or scales.dtype is not _bytes:
        raise TypeError(f"{what}: a checkpoint is int8 codes and uint8 scales")
    c, s = codes.shape, scales.shape
    if len(c) < 1 or len(s) != len(c) or c[:-1] != s[:-1] or s[-1] != (c[-1] + 31) // 32:
        raise ValueError(f"{what}: codes {tuple(c)} and scales {tuple(s)} are not one checkpoint")
    return codes, scales


def _kept(kept, t, shape, what):
    """(data, scales or None) of a tensor of type number t or a checkpoint, of the given shape."""
    if isinstance(kept, (tuple, list)):
        data, scales = _mx8(kept, what)
    else:
        data, scales = kept, None
        if data.dtype is not _dtypes[t]:
            raise TypeError(f"{what}: must be {_dtypes[t]} or a checkpoint")
    if data.shape != shape:
        raise ValueError(f"{what}: must have shape {tuple(shape)}")
    return data, scales


def mx8_quantize(x, codes=None, scales=None, stream=None):
    """The 8-bit checkpoint (codes int8 [..., K], scales uint8 [..., ceil(K / 32)]) of x
    [..., K] (bf16, float16 or float32; any K from 1 on)."""
    t = _type(x, "mx8_quantize")
    shape = x.shape
    if len(shape) < 1 or shape[-1] == 0:
        raise ValueError("mx8_quantize: the last dimension must not be empty")
    dev = _same_place("mx8_quantize", x)
    K, n, lead = shape[-1], x.numel(), shape[:-1]
    codes = _new(shape, _int8, x, dev) if codes is None else _out(codes, shape, _int8, x, "mx8_quantize codes")
    each = lead + ((K + 31) // 32,)
    scales = (_new(each, _bytes, x, dev) if scales is None
              else _out(scales, each, _bytes, x, "mx8_quantize scales"))
    if n:
        _call((_lib or lib()).swiglu_q_mx8_quantize, dev, stream, x.data_ptr(), n // K, K, t, codes.data_ptr(),
              scales.data_ptr())
    return codes, scales


def mx8_dequantize(codes, scales, dtype=None, out=None, stream=None):
    """The values [..., K] of a checkpoint, in bf16 (default), float16 or float32."""
    _mx8((codes, scales), "mx8_dequantize")
    dtype = _dtypes[0] if dtype is None else dtype
    dev = _same_place("mx8_dequantize", codes, scales)
    shape, n = codes.shape, codes.numel()
    out = _new(shape, dtype, codes, dev) if out is None else _out(out, shape, dtype, codes, "mx8_dequantize")
    t = _type(out, "mx8_dequantize")
    if n:
        _call((_lib or lib()).swiglu_q_mx8_dequantize, dev, stream, codes.data_ptr(), scales.data_ptr(),
              n // shape[-1], shape[-1], t, out.data_ptr())
    return out


def dense_linear(x, w, bias=None, act=SWQ_ACT_NONE, residual=None, keep=None, out_mode=None, out=None, stream=None):
    """``act(z) + residual``, ``z = x W^T + bias``, for x [..., K], W [N, K], bias [N] and residual
    [..., N], all bf16 or all float16.  Returns ``out`` [..., N] in x's type, or float32 with SWQ_LINEAR_F32; with
    keep the pair (out, z), z for ``dense_linear_backward``: keep="same" in x's type, keep="mx8" as
    a checkpoint (codes, scales).  x and w begin at multiples of 16 bytes.  Nothing is recorded for torch's backward pass, as
    of every function here: the caller asks for the gradients."""
    t = _type(x, "dense_linear", wide=False)
    if len(w.shape) != 2 or w.dtype != x.dtype or len(x.shape) < 1 or w.shape[1] != x.shape[-1]:
        raise ValueError(f"dense_linear: w must be {x.dtype} [N, K] with x's K")
    N, K = w.shape
    if K == 0 or N == 0:
        raise ValueError("dense_linear: a product needs inputs and outputs (K = 0 or N = 0)")
    if bias is not None and (bias.dtype != x.dtype or bias.shape != (N,)):
        raise ValueError(f"dense_linear: bias must be {x.dtype} [{N}]")
    mode = _out_mode(out_mode, t, "dense_linear")
    lead = x.shape[:-1]
    shape = lead + (N,)
    res = _residual(residual, x, shape, "dense_linear")
    dev = _same_place("dense_linear", x, w, bias, residual)
    out = _new(shape, _dtypes[mode], x, dev) if out is None else _out(out, shape, _dtypes[mode], x, "dense_linear")
    z = scales = None
    if keep == "same":
        kept = z = _new(shape, x.dtype, x, dev)
    elif keep == "mx8":
        kept = z, scales = _new(shape, _int8, x, dev), _new(lead + ((N + 31) // 32,), _bytes, x, dev)
    elif keep is not None:
        raise ValueError('dense_linear: keep must be None, "same" or "mx8"')
    n = x.numel()
    if n:
        _call((_lib or lib()).swiglu_q_dense_linear, dev, stream, x.data_ptr(), w.data_ptr(),
              None if bias is None else bias.data_ptr(), res, n // K, K, N, t, act, mode, out.data_ptr(),
              None if z is None else z.data_ptr(), None if scales is None else scales.data_ptr())
    return out if keep is None else (out, kept)


def dense_linear_backward(dout, x, w, z=None, act=SWQ_ACT_NONE, want=(True, True, True), dx=None, dw=None, dbias=None,
                          stream=None):
    """(dx [..., K], dw [N, K], dbias [N]) of ``dense_linear`` for dout [..., N], in dout's type (bf16 or
    float16); None where want says False.  x (needed for dw) and z (needed unless act is SWQ_ACT_NONE) are tensors
    of that type or checkpoints (codes, scales).  The residual's gradient is dout itself.  dout, w where dx is wanted and x
    where dw is begin at multiples of 16 bytes.  dz is rounded to dout's type for dx and dw (float16: past 65504 an infinity)."""
    t = _type(dout, "dense_linear_backward", wide=False)
    if len(w.shape) != 2 or w.dtype != dout.dtype or len(dout.shape) < 1 or w.shape[0] != dout.shape[-1]:
        raise ValueError(f"dense_linear_backward: w must be {dout.dtype} [N, K] with dout's N")
    N, K = w.shape
    if K == 0 or N == 0:
        raise ValueError("dense_linear_backward: a product needs inputs and outputs (K = 0 or N = 0)")
    want_x, want_w, want_b = want
    lead = dout.shape[:-1]
    xs = None
    if x is not None:
        x, xs = _kept(x, t, lead + (K,), "dense_linear_backward x")
    elif want_w:
        raise ValueError("dense_linear_backward: dw needs x")
    zs = None
    if z is not None:
        z, zs = _kept(z, t, dout.shape, "dense_linear_backward z")
    elif act != SWQ_ACT_NONE:
        raise ValueError("dense_linear_backward: an activation's gradient needs z")
    dev = _same_place("dense_linear_backward", dout, x, xs, w, z, zs)
    dtype = dout.dtype
    if not want_x:
        dx = None
    else:
        dx = (_new(lead + (K,), dtype, dout, dev) if dx is None
              else _out(dx, lead + (K,), dtype, dout, "dense_linear_backward dx"))
    if not want_w:
        dw = None
    else:
        dw = _new((N, K), dtype, dout, dev) if dw is None else _out(dw, (N, K), dtype, dout, "dense_linear_backward dw")
    if not want_b:
        dbias = None
    else:
        dbias = _new((N,), dtype, dout, dev) if dbias is None else _out(dbias, (N,), dtype, dout, "dense_linear_backward dbias")
    if want_x or want_w or want_b:
        n = dout.numel()
        # (with no rows the gradients of W and the bias are zeros; empty tensors have no address)
        at = [None if q is None else q.data_ptr() for q in (x, xs, z, zs, dx, dw, dbias)]
        if n:
            _call((_lib or lib()).swiglu_q_dense_linear_backward, dev, stream, dout.data_ptr(), at[0], at[1],
                  w.data_ptr(), at[2], at[3], n // N, K, N, t, act, *at[4:])
        elif want_w or want_b:
            none = 1 << 12                        # an address that is not read
            _call((_lib or lib()).swiglu_q_dense_linear_backward, dev, stream, none, none, None, none, none, None, 0, K,
                  N, t, act, None, *at[5:])
    return dx, dw, dbias


def swiglu(gate, up, keep=False, hidden=None, stream=None):
    """``silu(gate) * up`` for gate and up [..., K] (bf16 or float16).  With keep the triple (hidden, gate,
    up), gate and up as checkpoints for ``swiglu_backward``, which is the caller's to call: nothing is recorded for torch's
    backward pass."""
    t = _type(gate, "swiglu", wide=False)
    shape = gate.shape
    if up.dtype != gate.dtype or up.shape != shape or len(shape) < 1 or shape[-1] == 0:
        raise ValueError("swiglu: gate and up must be of one type and shape [..., K], K from 1 on")
    dev = _same_place("swiglu", gate, up)
    hidden = _new(shape, gate.dtype, gate, dev) if hidden is None else _out(hidden, shape, gate.dtype, gate, "swiglu hidden")
    K, n = shape[-1], gate.numel()
    at = (None,) * 4
    if keep:
        each = shape[:-1] + ((K + 31) // 32,)
        gc, uc = _several(shape, (_int8, _int8), gate, dev)
        gs, us = _several(each, (_bytes, _bytes), gate, dev)
        at = (gc.data_ptr(), gs.data_ptr(), uc.data_ptr(), us.data_ptr())
    if n:
        _call((_lib or lib()).swiglu_q_swiglu, dev, stream, gate.data_ptr(), up.data_ptr(), n // K, K, t,
              hidden.data_ptr(), *at)
    return (hidden, (gc, gs), (uc, us)) if keep else hidden


def swiglu_backward(dhidden, gate, up, hidden=False, stream=None):
    """(dgate, dup) of ``swiglu`` for dhidden [..., K] (bf16 or float16), with hidden=True the triple (dgate, dup,
    hidden).  gate and up are tensors of that type or checkpoints; from checkpoints the gradients and hidden are those of the
    values that these hold, not of the tensors that they were made from."""
    t = _type(dhidden, "swiglu_backward", wide=False)
    shape = dhidden.shape
    if len(shape) < 1 or shape[-1] == 0:
        raise ValueError("swiglu_backward: dhidden must be [..., K], K from 1 on")
    gate, gs = _kept(gate, t, shape, "swiglu_backward gate")
    up, us = _kept(up, t, shape, "swiglu_backward up")
    dev = _same_place("swiglu_backward", dhidden, gate, gs, up, us)
    outs = _several(shape, (dhidden.dtype,) * (3 if hidden else 2), dhidden, dev)
    K, n = shape[-1], dhidden.numel()
    if n:
        _call((_lib or lib()).swiglu_q_swiglu_backward, dev, stream, dhidden.data_ptr(), gate.data_ptr(),
              None if gs is None else gs.data_ptr(), up.data_ptr(), None if us is None else us.data_ptr(), n // K, K, t,
              outs[0].data_ptr(), outs[1].data_ptr(), outs[2].data_ptr() if hidden else None)
    return tuple(outs)


def _slots(logits, ids, what):
    """(T, E, k) of logits [..., E] and ids [..., k]."""
    if len(logits.shape) < 1 or ids.dtype != _int32 or len(ids.shape) < 1 or ids.shape[:-1] != logits.shape[:-1]:
        raise ValueError(f"{what}: ids must be int32 [..., k] with the logits' leading shape")
    E, k = logits.shape[-1], ids.shape[-1]
    return logits.shape[:-1].numel(), E, k


def balance_loss(logits, ids, scoring=SWQ_ROUTE_SOFTMAX, stream=None):
    """(loss float32 [], counts int32 [E], slopes float32 [E]) of a router's choice: logits [..., E] and
    ``route``'s ids [..., k].  The loss is ``E sum_e f_e P_e``, f_e the expert's share of the slots, P_e its mean
    probability over the tokens with a slot; counts are the experts' slots, slopes go to ``route_backward``."""
    t = _type(logits, "balance_loss")
    T, E, k = _slots(logits, ids, "balance_loss")
    dev = _same_place("balance_loss", logits, ids)
    loss = _new((), _float32, logits, dev)
    counts, slopes = _several((E,), (_int32, _float32), logits, dev)
    at = loss.data_ptr()
    _call((_lib or lib()).swiglu_q_balance_loss, dev, stream, logits.data_ptr() if T else at,
          ids.data_ptr() if T else at, T, E, k, t, scoring, at, counts.data_ptr(), slopes.data_ptr())
    return loss, counts, slopes


def route_backward(logits, ids, dweights=None, scoring=SWQ_ROUTE_SOFTMAX, slopes=None, dloss=None, dlogits=None,
                   stream=None):
    """dlogits [..., E] in the logits' type: the gradient of ``route``'s weights for ids, given theirs (dweights
    float32 [..., k]), and of ``balance_loss``, given its slopes and its own gradient dloss (float32, one
    value on the GPU; None: 1).  Either may be left out, not both."""
    t = _type(logits, "route_backward")
    T, E, k = _slots(logits, ids, "route_backward")
    if dweights is None and slopes is None:
        raise ValueError("route_backward: needs dweights or slopes")
    if dweights is not None and (dweights.dtype != _float32 or dweights.shape != ids.shape):
        raise ValueError("route_backward: dweights must be float32 of ids' shape")
    if slopes is not None and (slopes.dtype != _float32 or slopes.shape != (E,)):
        raise ValueError(f"route_backward: slopes must be float32 [{E}]")
    if dloss is not None and (slopes is None or dloss.dtype != _float32 or dloss.numel() != 1):
        raise ValueError("route_backward: dloss must be one float32 beside slopes")
    dev = _same_place("route_backward", logits, ids, dweights, slopes, dloss)
    shape = logits.shape
    dlogits = (_new(shape, logits.dtype, logits, dev) if dlogits is None
               else _out(dlogits, shape, logits.dtype, logits, "route_backward dlogits"))
    if T and E:
        _call((_lib or lib()).swiglu_q_route_backward, dev, stream, logits.data_ptr(), ids.data_ptr(),
              None if dweights is None else dweights.data_ptr(), None if slopes is None else slopes.data_ptr(),
              None if dloss is None else dloss.data_ptr(), T, E, k, t, scoring, dlogits.data_ptr())
    return dlogits


def debug_gemm_tensors(x, wg, sg, bg, wu, su, bu, bits_g, gs_g, bits_u=None, gs_u=None,
                       path=SWQ_PATH_AUTO, stream=None):
    """Pre-epilogue float32 (gate, up) from the kernel of ``path``."""
    import torch
    bits_u = bits_g if bits_u is None else bits_u
    gs_u = gs_g if gs_u is None else gs_u
    x, _ = _rows(x, "debug_gemm")
    M, H = int(x.shape[0]), int(x.shape[1])
    I = int(wg.shape[0])
    g = torch.empty((M, I), dtype=torch.float32, device=x.device)
    u = torch.empty((M, I), dtype=torch.float32, device=x.device)
    rc = swiglu_q_debug_gemm(x, wg, sg, bg, wu, su, bu, M, H, I, bits_g, gs_g, bits_u, gs_u, path, g, u, stream)
    if rc != SWQ_OK:
        raise SwigluQError(rc, "swiglu_q_debug_gemm")
    return g, u


def to_device(prob, device="cuda"):
    """Copy a host problem (numpy bit patterns) to device tensors; returns the
    tuple (x, wg, sg, bg, wu, su, bu), x and the scales and biases as bf16, or
    float16 for a problem drawn with binary16 activations."""
    import numpy as np
    import torch
    dt16 = torch.float16 if getattr(prob, "act", "bf16") == "f16" else torch.bfloat16

    def t16(a):
        return torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).to(device).view(dt16)

    def t32(a):
        return torch.from_numpy(np.ascontiguousarray(a).view(np.int32)).to(device)

    return (t16(prob.x), t32(prob.wg), t16(prob.sg), t16(prob.bg),
            t32(prob.wu), t16(prob.su), t16(prob.bu))
