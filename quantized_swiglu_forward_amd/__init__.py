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
_bytes = _int32 = _float32 = None
_raw_stream = _device_now = _on_device = None   # torch's current stream of a GPU, current GPU, GPU guard


def _load_types():
    global _types, _dtypes, _words, _bytes, _int32, _float32, _raw_stream, _device_now, _on_device
    import torch
    _dtypes = (torch.bfloat16, torch.float32, torch.float16)
    _words = (torch.int32, torch.uint32)
    _bytes, _int32, _float32 = torch.uint8, torch.int32, torch.float32
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda dev: torch.cuda.current_stream(dev).cuda_stream)
    _device_now = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    _on_device = torch.cuda.device
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
