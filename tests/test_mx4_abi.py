"""The MXFP4 operators, the router and the experts' MLP without a GPU: bad
arguments are rejected before any HIP call, by status in C and by exception in
the tensor functions; and the reference quantiser that the GPU tests use is
held to values written out by hand."""
import numpy as np
import pytest
import torch

import mx4_reference as ref
import quantized_swiglu_forward_amd as swq

P = 1 << 20    # a fake, aligned "device" address: validation never dereferences it
NULL, SHAPE, UNSUP, ALIGN, OK = (swq.SWQ_ERR_NULL, swq.SWQ_ERR_SHAPE, swq.SWQ_ERR_UNSUPPORTED, swq.SWQ_ERR_ALIGN,
                                 swq.SWQ_OK)

QUANT = dict(x=P, R=4, K=64, type=0, codes=P, scales=P, stream=0)
DEQUANT = dict(codes=P, scales=P, R=4, K=64, type=0, out=P, stream=0)
LINEAR = dict(x=P, W=P, s=P, residual=None, M=4, K=64, N=8, type=0, out_mode=0, out=P, stream=0)
MATMUL = dict(A=P, sa=P, W=P, sw=P, M=4, K=64, N=8, out_mode=0, out=P, stream=0)
GROUPED = dict(x=P, offsets=P, W=P, s=P, P=4, E=3, K=64, N=8, type=0, out_mode=0, out=P, stream=0)
ROUTE = dict(logits=P, T=4, E=8, k=2, type=0, scoring=0, ids=P, weights=P, stream=0)
MOE = dict(x=P, ids=P, weights=P, Wg=P, sg=P, Wu=P, su=P, Wd=P, sd=P, residual=None, T=4, k=2, E=8, H=64, I=32, Ho=64,
           type=0, out_mode=0, out=P, stream=0)


@pytest.mark.parametrize("fn,base,kw,status", [
    (swq.swiglu_q_mx4_quantize, QUANT, dict(x=None), NULL),
    (swq.swiglu_q_mx4_quantize, QUANT, dict(codes=None), NULL),
    (swq.swiglu_q_mx4_quantize, QUANT, dict(scales=None), NULL),
    (swq.swiglu_q_mx4_quantize, QUANT, dict(type=3), UNSUP),
    (swq.swiglu_q_mx4_quantize, QUANT, dict(K=48), SHAPE),
    (swq.swiglu_q_mx4_quantize, QUANT, dict(K=0), SHAPE),
    (swq.swiglu_q_mx4_quantize, QUANT, dict(R=-1), SHAPE),
    (swq.swiglu_q_mx4_quantize, QUANT, dict(R=1 << 30, K=1 << 20), SHAPE),
    (swq.swiglu_q_mx4_quantize, QUANT, dict(x=P + 8), ALIGN),
    (swq.swiglu_q_mx4_quantize, QUANT, dict(codes=P + 4), ALIGN),
    (swq.swiglu_q_mx4_quantize, QUANT, dict(R=0), OK),
    (swq.swiglu_q_mx4_dequantize, DEQUANT, dict(codes=None), NULL),
    (swq.swiglu_q_mx4_dequantize, DEQUANT, dict(out=None), NULL),
    (swq.swiglu_q_mx4_dequantize, DEQUANT, dict(type=-1), UNSUP),
    (swq.swiglu_q_mx4_dequantize, DEQUANT, dict(K=33), SHAPE),
    (swq.swiglu_q_mx4_dequantize, DEQUANT, dict(out=P + 8), ALIGN),
    (swq.swiglu_q_mx4_dequantize, DEQUANT, dict(R=0), OK),
    (swq.swiglu_q_mx4_linear, LINEAR, dict(x=None), NULL),
    (swq.swiglu_q_mx4_linear, LINEAR, dict(W=None), NULL),
    (swq.swiglu_q_mx4_linear, LINEAR, dict(s=None), NULL),
    (swq.swiglu_q_mx4_linear, LINEAR, dict(out=None), NULL),
    (swq.swiglu_q_mx4_linear, LINEAR, dict(type=1), UNSUP),
    (swq.swiglu_q_mx4_linear, LINEAR, dict(out_mode=2), UNSUP),
    (swq.swiglu_q_mx4_linear, LINEAR, dict(type=2, out_mode=0), UNSUP),
    (swq.swiglu_q_mx4_linear, LINEAR, dict(M=-1), SHAPE),
    (swq.swiglu_q_mx4_linear, LINEAR, dict(K=40), SHAPE),
    (swq.swiglu_q_mx4_linear, LINEAR, dict(N=0), SHAPE),
    (swq.swiglu_q_mx4_linear, LINEAR, dict(M=1 << 30, N=1 << 30), SHAPE),
    (swq.swiglu_q_mx4_linear, LINEAR, dict(x=P + 2), ALIGN),
    (swq.swiglu_q_mx4_linear, LINEAR, dict(W=P + 4), ALIGN),
    (swq.swiglu_q_mx4_linear, LINEAR, dict(out=P + 1), ALIGN),
    (swq.swiglu_q_mx4_linear, LINEAR, dict(out=P + 2, out_mode=1), ALIGN),
    (swq.swiglu_q_mx4_linear, LINEAR, dict(residual=P + 1), ALIGN),
    (swq.swiglu_q_mx4_linear, LINEAR, dict(M=0), OK),
    (swq.swiglu_q_mx4_matmul, MATMUL, dict(A=None), NULL),
    (swq.swiglu_q_mx4_matmul, MATMUL, dict(sw=None), NULL),
    (swq.swiglu_q_mx4_matmul, MATMUL, dict(out_mode=3), UNSUP),
    (swq.swiglu_q_mx4_matmul, MATMUL, dict(K=16), SHAPE),
    (swq.swiglu_q_mx4_matmul, MATMUL, dict(A=P + 8), ALIGN),
    (swq.swiglu_q_mx4_matmul, MATMUL, dict(M=0), OK),
    (swq.swiglu_q_mx4_grouped_linear, GROUPED, dict(offsets=None), NULL),
    (swq.swiglu_q_mx4_grouped_linear, GROUPED, dict(E=0), SHAPE),
    (swq.swiglu_q_mx4_grouped_linear, GROUPED, dict(E=1025), SHAPE),
    (swq.swiglu_q_mx4_grouped_linear, GROUPED, dict(offsets=P + 2), ALIGN),
    (swq.swiglu_q_mx4_grouped_linear, GROUPED, dict(type=1), UNSUP),
    (swq.swiglu_q_mx4_grouped_linear, GROUPED, dict(P=0), OK),
    (swq.swiglu_q_route, ROUTE, dict(logits=None), NULL),
    (swq.swiglu_q_route, ROUTE, dict(ids=None), NULL),
    (swq.swiglu_q_route, ROUTE, dict(k=0), SHAPE),
    (swq.swiglu_q_route, ROUTE, dict(k=9), SHAPE),
    (swq.swiglu_q_route, ROUTE, dict(E=1025), SHAPE),
    (swq.swiglu_q_route, ROUTE, dict(E=200, k=65), SHAPE),
    (swq.swiglu_q_route, ROUTE, dict(scoring=4), UNSUP),
    (swq.swiglu_q_route, ROUTE, dict(type=5), UNSUP),
    (swq.swiglu_q_route, ROUTE, dict(weights=P + 2), ALIGN),
    (swq.swiglu_q_route, ROUTE, dict(T=0), OK),
    (swq.swiglu_q_moe_mlp, MOE, dict(ids=None), NULL),
    (swq.swiglu_q_moe_mlp, MOE, dict(sd=None), NULL),
    (swq.swiglu_q_moe_mlp, MOE, dict(k=0), SHAPE),
    (swq.swiglu_q_moe_mlp, MOE, dict(E=0), SHAPE),
    (swq.swiglu_q_moe_mlp, MOE, dict(H=65), SHAPE),
    (swq.swiglu_q_moe_mlp, MOE, dict(I=16), SHAPE),
    (swq.swiglu_q_moe_mlp, MOE, dict(Ho=0), SHAPE),
    (swq.swiglu_q_moe_mlp, MOE, dict(T=1 << 30, k=2), SHAPE),
    (swq.swiglu_q_moe_mlp, MOE, dict(Wu=P + 4), ALIGN),
    (swq.swiglu_q_moe_mlp, MOE, dict(type=1), UNSUP),
    (swq.swiglu_q_moe_mlp, MOE, dict(T=0), OK),
])
def test_status(fn, base, kw, status):
    assert fn(**{**base, **kw}) == status


def _mx(*shape):
    return torch.zeros(*shape[:-1], shape[-1] // 8, dtype=torch.int32), torch.zeros(*shape[:-1], shape[-1] // 32,
                                                                                     dtype=torch.uint8)


@pytest.mark.parametrize("call,error", [
    (lambda: swq.mx4_quantize(torch.zeros(2, 48)), ValueError),
    (lambda: swq.mx4_quantize(torch.zeros(2, 64, dtype=torch.float64)), TypeError),
    (lambda: swq.mx4_quantize(torch.zeros(64, 2).t()), ValueError),
    (lambda: swq.mx4_quantize(torch.zeros(2, 64)), ValueError),                       # not on a GPU
    (lambda: swq.mx4_dequantize(torch.zeros(2, 8, dtype=torch.int64), torch.zeros(2, 2, dtype=torch.uint8)), TypeError),
    (lambda: swq.mx4_dequantize(torch.zeros(2, 8, dtype=torch.int32), torch.zeros(2, 3, dtype=torch.uint8)), ValueError),
    (lambda: swq.mx4_linear(torch.zeros(2, 64), *_mx(8, 64)), TypeError),             # float32 activations
    (lambda: swq.mx4_linear(torch.zeros(2, 96).bfloat16(), *_mx(8, 64)), ValueError),
    (lambda: swq.mx4_linear(torch.zeros(2, 64).bfloat16(), *_mx(8, 64), out_mode=swq.SWQ_LINEAR_F16), ValueError),
    (lambda: swq.mx4_linear(torch.zeros(2, 64).bfloat16(), *_mx(8, 64), residual=torch.zeros(2, 8)), ValueError),
    (lambda: swq.mx4_matmul(*_mx(2, 96), *_mx(8, 64)), ValueError),
    (lambda: swq.mx4_matmul(*_mx(2, 64), *_mx(8, 64), out_mode=7), ValueError),
    (lambda: swq.mx4_grouped_linear(torch.zeros(2, 64).bfloat16(), torch.zeros(3, dtype=torch.int32), *_mx(3, 8, 64)),
     ValueError),
    (lambda: swq.mx4_grouped_linear(torch.zeros(2, 64).bfloat16(), torch.zeros(4, dtype=torch.int64), *_mx(3, 8, 64)),
     ValueError),
    (lambda: swq.route(torch.zeros(2, 8, dtype=torch.int32), 2), TypeError),
    (lambda: swq.route(torch.zeros(2, 8), 2), ValueError),                            # not on a GPU
    (lambda: swq.moe_mlp(torch.zeros(2, 64).bfloat16(), torch.zeros(2, 2, dtype=torch.int64), torch.zeros(2, 2),
                         *_mx(4, 32, 64), *_mx(4, 32, 64), *_mx(4, 64, 32)), ValueError),
    (lambda: swq.moe_mlp(torch.zeros(2, 64).bfloat16(), torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, 2),
                         *_mx(4, 32, 64), *_mx(4, 32, 64), *_mx(3, 64, 32)), ValueError),
    (lambda: swq.moe_mlp(torch.zeros(2, 64).bfloat16(), torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, 2),
                         *_mx(4, 32, 64), *_mx(4, 64, 64), *_mx(4, 64, 32)), ValueError),
])
def test_tensor_functions_refuse(call, error):
    with pytest.raises(error):
        call()


def test_reference_quantiser():
    """Ties to even, saturation, clamped scales, signed zeros, NaN blocks."""
    x = torch.zeros(6, 32)
    x[0, :8] = torch.tensor([4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, -5.0])
    x[1, :4] = torch.tensor([7.9, 5.01, -0.26, -0.0])
    x[2, :2] = torch.tensor([2.0 ** -126, 2.0 ** -149])
    x[3, 3] = float("inf")
    x[4, 0] = 2.0 ** 127
    codes, scales = ref.quantize(x)
    assert codes[0, :8].tolist() == [6, 0, 2, 2, 4, 4, 6, 14] and scales[0, 0] == 127
    assert codes[1, :4].tolist() == [7, 7, 9, 8] and scales[1, 0] == 127
    assert codes[2, :2].tolist() == [4, 0] and scales[2, 0] == 0
    assert scales[3, 0] == 255 and not codes[3].any()
    assert codes[4, 0] == 6 and scales[4, 0] == 252
    assert scales[5, 0] == 0 and not codes[5].any()


def test_reference_values():
    codes = torch.tensor([[0x76543210, -0x01234568, 0, 0]], dtype=torch.int32)     # second word 0xFEDCBA98
    v = ref.values(codes, torch.tensor([[128]], dtype=torch.uint8))
    assert v[0, :8].tolist() == [0, 1, 2, 3, 4, 6, 8, 12]
    assert v[0, 8:16].tolist() == [0, -1, -2, -3, -4, -6, -8, -12]
    assert np.isnan(ref.values(codes, torch.tensor([[255]], dtype=torch.uint8))).all()
