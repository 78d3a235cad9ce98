"""The products with 16-bit weights, the checkpoints, the SwiGLU with
checkpoints and the router's loss and gradient without a GPU: bad arguments are
rejected before any HIP call, by status in C and by exception in the tensor
functions; and the 64-bit reference that the GPU tests use is held to values
written out by hand."""
import numpy as np
import pytest
import torch

import dense_reference as ref
import quantized_swiglu_forward_amd as swq

P = 1 << 20    # a fake, aligned "device" address: validation never dereferences it
NULL, SHAPE, UNSUP, ALIGN, OK = (swq.SWQ_ERR_NULL, swq.SWQ_ERR_SHAPE, swq.SWQ_ERR_UNSUPPORTED, swq.SWQ_ERR_ALIGN,
                                 swq.SWQ_OK)

QUANT = dict(x=P, R=4, K=64, type=0, codes=P, scales=P, stream=0)
DEQUANT = dict(codes=P, scales=P, R=4, K=64, type=0, out=P, stream=0)
LINEAR = dict(x=P, W=P, bias=P, residual=P, M=4, K=60, N=9, type=0, act=2, out_mode=0, out=P, z=P, z_scales=P, stream=0)
BACK = dict(dout=P, x=P, x_scales=P, W=P, z=P, z_scales=P, M=4, K=60, N=9, type=0, act=2, dx=P, dW=P, dbias=P, stream=0)
SWIGLU = dict(gate=P, up=P, R=4, K=60, type=0, hidden=P, gate_codes=P, gate_scales=P, up_codes=P, up_scales=P, stream=0)
SWIGLU_B = dict(dhidden=P, gate=P, gate_scales=P, up=P, up_scales=P, R=4, K=60, type=0, dgate=P, dup=P, hidden=P, stream=0)
BALANCE = dict(logits=P, ids=P, T=4, E=8, k=2, type=0, scoring=0, loss=P, counts=P, slopes=P, stream=0)
ROUTE_B = dict(logits=P, ids=P, dweights=P, slopes=P, dloss=P, T=4, E=8, k=2, type=0, scoring=0, dlogits=P, stream=0)


@pytest.mark.parametrize("fn,base,kw,status", [
    (swq.swiglu_q_mx8_quantize, QUANT, dict(x=None), NULL),
    (swq.swiglu_q_mx8_quantize, QUANT, dict(codes=None), NULL),
    (swq.swiglu_q_mx8_quantize, QUANT, dict(scales=None), NULL),
    (swq.swiglu_q_mx8_quantize, QUANT, dict(type=3), UNSUP),
    (swq.swiglu_q_mx8_quantize, QUANT, dict(K=0), SHAPE),
    (swq.swiglu_q_mx8_quantize, QUANT, dict(R=-1), SHAPE),
    (swq.swiglu_q_mx8_quantize, QUANT, dict(R=1 << 30, K=1 << 20), SHAPE),
    (swq.swiglu_q_mx8_quantize, QUANT, dict(K=(1 << 20) + 1), SHAPE),
    (swq.swiglu_q_mx8_quantize, QUANT, dict(x=P + 1), ALIGN),
    (swq.swiglu_q_mx8_quantize, QUANT, dict(x=P + 2, type=1), ALIGN),
    (swq.swiglu_q_mx8_quantize, QUANT, dict(R=0), OK),
    (swq.swiglu_q_mx8_dequantize, DEQUANT, dict(scales=None), NULL),
    (swq.swiglu_q_mx8_dequantize, DEQUANT, dict(out=None), NULL),
    (swq.swiglu_q_mx8_dequantize, DEQUANT, dict(type=-1), UNSUP),
    (swq.swiglu_q_mx8_dequantize, DEQUANT, dict(out=P + 1), ALIGN),
    (swq.swiglu_q_mx8_dequantize, DEQUANT, dict(R=0), OK),
    (swq.swiglu_q_dense_linear, LINEAR, dict(x=None), NULL),
    (swq.swiglu_q_dense_linear, LINEAR, dict(W=None), NULL),
    (swq.swiglu_q_dense_linear, LINEAR, dict(out=None), NULL),
    (swq.swiglu_q_dense_linear, LINEAR, dict(z=None), NULL),                 # scales without codes
    (swq.swiglu_q_dense_linear, LINEAR, dict(type=1), UNSUP),
    (swq.swiglu_q_dense_linear, LINEAR, dict(act=5), UNSUP),
    (swq.swiglu_q_dense_linear, LINEAR, dict(act=-1), UNSUP),
    (swq.swiglu_q_dense_linear, LINEAR, dict(out_mode=2), UNSUP),
    (swq.swiglu_q_dense_linear, LINEAR, dict(M=-1), SHAPE),
    (swq.swiglu_q_dense_linear, LINEAR, dict(K=0), SHAPE),
    (swq.swiglu_q_dense_linear, LINEAR, dict(N=0), SHAPE),
    (swq.swiglu_q_dense_linear, LINEAR, dict(N=(1 << 20) + 1), SHAPE),
    (swq.swiglu_q_dense_linear, LINEAR, dict(M=(1 << 30) + 1), SHAPE),
    (swq.swiglu_q_dense_linear, LINEAR, dict(x=P + 8), ALIGN),
    (swq.swiglu_q_dense_linear, LINEAR, dict(W=P + 2), ALIGN),
    (swq.swiglu_q_dense_linear, LINEAR, dict(bias=P + 1), ALIGN),
    (swq.swiglu_q_dense_linear, LINEAR, dict(residual=P + 1), ALIGN),
    (swq.swiglu_q_dense_linear, LINEAR, dict(out=P + 2, out_mode=1), ALIGN),
    (swq.swiglu_q_dense_linear, LINEAR, dict(z=P + 1, z_scales=None), ALIGN),
    (swq.swiglu_q_dense_linear, LINEAR, dict(M=0), OK),
    (swq.swiglu_q_dense_linear_backward, BACK, dict(dout=None), NULL),
    (swq.swiglu_q_dense_linear_backward, BACK, dict(dx=None, dW=None, dbias=None), NULL),
    (swq.swiglu_q_dense_linear_backward, BACK, dict(W=None), NULL),
    (swq.swiglu_q_dense_linear_backward, BACK, dict(x=None), NULL),
    (swq.swiglu_q_dense_linear_backward, BACK, dict(z=None), NULL),
    (swq.swiglu_q_dense_linear_backward, BACK, dict(type=1), UNSUP),
    (swq.swiglu_q_dense_linear_backward, BACK, dict(act=9), UNSUP),
    (swq.swiglu_q_dense_linear_backward, BACK, dict(K=0), SHAPE),
    (swq.swiglu_q_dense_linear_backward, BACK, dict(M=-1), SHAPE),
    (swq.swiglu_q_dense_linear_backward, BACK, dict(dout=P + 8), ALIGN),
    (swq.swiglu_q_dense_linear_backward, BACK, dict(x=P + 8, x_scales=None), ALIGN),
    (swq.swiglu_q_dense_linear_backward, BACK, dict(z=P + 1, z_scales=None), ALIGN),
    (swq.swiglu_q_dense_linear_backward, BACK, dict(dW=P + 1), ALIGN),
    (swq.swiglu_q_swiglu, SWIGLU, dict(gate=None), NULL),
    (swq.swiglu_q_swiglu, SWIGLU, dict(hidden=None), NULL),
    (swq.swiglu_q_swiglu, SWIGLU, dict(up_scales=None), NULL),               # all four or none
    (swq.swiglu_q_swiglu, SWIGLU, dict(type=1), UNSUP),
    (swq.swiglu_q_swiglu, SWIGLU, dict(K=0), SHAPE),
    (swq.swiglu_q_swiglu, SWIGLU, dict(up=P + 1), ALIGN),
    (swq.swiglu_q_swiglu, SWIGLU, dict(R=0), OK),
    (swq.swiglu_q_swiglu_backward, SWIGLU_B, dict(dhidden=None), NULL),
    (swq.swiglu_q_swiglu_backward, SWIGLU_B, dict(dup=None), NULL),
    (swq.swiglu_q_swiglu_backward, SWIGLU_B, dict(type=1), UNSUP),
    (swq.swiglu_q_swiglu_backward, SWIGLU_B, dict(R=-1), SHAPE),
    (swq.swiglu_q_swiglu_backward, SWIGLU_B, dict(gate=P + 1, gate_scales=None), ALIGN),
    (swq.swiglu_q_swiglu_backward, SWIGLU_B, dict(dgate=P + 1), ALIGN),
    (swq.swiglu_q_swiglu_backward, SWIGLU_B, dict(R=0), OK),
    (swq.swiglu_q_balance_loss, BALANCE, dict(ids=None), NULL),
    (swq.swiglu_q_balance_loss, BALANCE, dict(loss=None), NULL),
    (swq.swiglu_q_balance_loss, BALANCE, dict(slopes=None), NULL),
    (swq.swiglu_q_balance_loss, BALANCE, dict(type=4), UNSUP),
    (swq.swiglu_q_balance_loss, BALANCE, dict(scoring=4), UNSUP),
    (swq.swiglu_q_balance_loss, BALANCE, dict(E=1025), SHAPE),
    (swq.swiglu_q_balance_loss, BALANCE, dict(k=0), SHAPE),
    (swq.swiglu_q_balance_loss, BALANCE, dict(k=65), SHAPE),
    (swq.swiglu_q_balance_loss, BALANCE, dict(T=1 << 30, k=2), SHAPE),
    (swq.swiglu_q_balance_loss, BALANCE, dict(logits=P + 2, type=1), ALIGN),
    (swq.swiglu_q_balance_loss, BALANCE, dict(counts=P + 2), ALIGN),
    (swq.swiglu_q_route_backward, ROUTE_B, dict(logits=None), NULL),
    (swq.swiglu_q_route_backward, ROUTE_B, dict(dweights=None, slopes=None, dloss=None), NULL),
    (swq.swiglu_q_route_backward, ROUTE_B, dict(slopes=None), NULL),         # dloss without slopes
    (swq.swiglu_q_route_backward, ROUTE_B, dict(scoring=-1), UNSUP),
    (swq.swiglu_q_route_backward, ROUTE_B, dict(E=0), SHAPE),
    (swq.swiglu_q_route_backward, ROUTE_B, dict(T=-1), SHAPE),
    (swq.swiglu_q_route_backward, ROUTE_B, dict(dlogits=P + 1), ALIGN),
    (swq.swiglu_q_route_backward, ROUTE_B, dict(dweights=P + 2), ALIGN),
    (swq.swiglu_q_route_backward, ROUTE_B, dict(T=0), OK),
])
def test_status(fn, base, kw, status):
    assert fn(**{**base, **kw}) == status


B = torch.bfloat16


def z(*shape, dtype=B):
    return torch.zeros(*shape, dtype=dtype)


def cp(*shape):
    return z(*shape, dtype=torch.int8), z(*shape[:-1], (shape[-1] + 31) // 32, dtype=torch.uint8)


@pytest.mark.parametrize("call,error", [
    (lambda: swq.mx8_quantize(z(2, 0)), ValueError),
    (lambda: swq.mx8_quantize(z(2, 8, dtype=torch.float64)), TypeError),
    (lambda: swq.mx8_quantize(z(8, 2).t()), ValueError),
    (lambda: swq.mx8_quantize(z(2, 8)), ValueError),                                   # not on a GPU
    (lambda: swq.mx8_dequantize(z(2, 8, dtype=torch.uint8), z(2, 1, dtype=torch.uint8)), TypeError),
    (lambda: swq.mx8_dequantize(z(2, 33, dtype=torch.int8), z(2, 1, dtype=torch.uint8)), ValueError),
    (lambda: swq.dense_linear(z(2, 8, dtype=torch.float32), z(3, 8)), TypeError),
    (lambda: swq.dense_linear(z(2, 8), z(3, 9)), ValueError),
    (lambda: swq.dense_linear(z(2, 8), z(3, 8, dtype=torch.float16)), ValueError),
    (lambda: swq.dense_linear(z(2, 0), z(3, 0)), ValueError),
    (lambda: swq.dense_linear(z(2, 8), z(0, 8)), ValueError),
    (lambda: swq.dense_linear(z(2, 8), z(3, 8), bias=z(2)), ValueError),
    (lambda: swq.dense_linear(z(2, 8), z(3, 8), residual=z(2, 2)), ValueError),
    (lambda: swq.dense_linear(z(2, 8), z(3, 8), out_mode=swq.SWQ_LINEAR_F16), ValueError),
    (lambda: swq.dense_linear(z(2, 8), z(3, 8)), ValueError),                          # not on a GPU
    (lambda: swq.dense_linear_backward(z(2, 3), z(2, 8), z(4, 8)), ValueError),
    (lambda: swq.dense_linear_backward(z(2, 3), z(2, 7), z(3, 8)), ValueError),
    (lambda: swq.dense_linear_backward(z(2, 3), z(2, 8, dtype=torch.float16), z(3, 8)), TypeError),
    (lambda: swq.dense_linear_backward(z(2, 3), z(2, 8), z(3, 8), act=swq.SWQ_ACT_SILU), ValueError),
    (lambda: swq.dense_linear_backward(z(2, 3), z(2, 8), z(3, 8), cp(2, 4), act=swq.SWQ_ACT_SILU), ValueError),
    (lambda: swq.dense_linear_backward(z(2, 3), (z(2, 8), z(2, 1)), z(3, 8)), TypeError),
    (lambda: swq.dense_linear_backward(z(2, 3), cp(2, 8), z(3, 8)), ValueError),       # not on a GPU
    (lambda: swq.swiglu(z(2, 8), z(2, 9)), ValueError),
    (lambda: swq.swiglu(z(2, 8), z(2, 8, dtype=torch.float16)), ValueError),
    (lambda: swq.swiglu(z(2, 8, dtype=torch.float32), z(2, 8, dtype=torch.float32)), TypeError),
    (lambda: swq.swiglu_backward(z(2, 8), cp(2, 8), z(2, 9)), ValueError),
    (lambda: swq.swiglu_backward(z(2, 8), cp(2, 8), cp(2, 8)), ValueError),            # not on a GPU
    (lambda: swq.balance_loss(z(2, 8), z(2, 2, dtype=torch.int64)), ValueError),
    (lambda: swq.balance_loss(z(2, 8), z(3, 2, dtype=torch.int32)), ValueError),
    (lambda: swq.balance_loss(z(2, 8), z(2, 2, dtype=torch.int32)), ValueError),       # not on a GPU
    (lambda: swq.route_backward(z(2, 8), z(2, 2, dtype=torch.int32)), ValueError),
    (lambda: swq.route_backward(z(2, 8), z(2, 2, dtype=torch.int32), z(2, 2)), ValueError),
    (lambda: swq.route_backward(z(2, 8), z(2, 2, dtype=torch.int32), slopes=z(7, dtype=torch.float32)), ValueError),
    (lambda: swq.route_backward(z(2, 8), z(2, 2, dtype=torch.int32), z(2, 2, dtype=torch.float32),
                                dloss=z(1, dtype=torch.float32)), ValueError),
])
def test_tensor_functions_refuse(call, error):
    with pytest.raises(error):
        call()


def test_reference_checkpoint():
    """Ties to even, the step's border, a short last block, NaN blocks, the smallest step."""
    x = torch.zeros(4, 34)
    x[0, :6] = torch.tensor([64.0, 0.5, 1.5, 2.5, -0.5, 63.49])
    x[0, 32:] = torch.tensor([127.5, 1.0])
    x[1, 3] = float("inf")
    x[2, 0] = 2.0 ** -149
    codes, scales = ref.mx8(x)
    assert codes[0, :6].tolist() == [64, 0, 2, 2, 0, 63] and scales[0].tolist() == [133, 134]
    assert codes[0, 32:].tolist() == [64, 0]                       # in steps of 2: 63.75, 0.5
    assert scales[1, 0] == 255 and not codes[1].any()
    assert scales[2, 0] == 7 and not codes[2].any() and scales[3, 0] == 7
    v = ref.mx8_values(torch.from_numpy(codes), torch.from_numpy(scales))
    assert v[0, 0] == 64.0 and v[0, 32] == 128.0 and torch.isnan(v[1, :32]).all()
    assert np.allclose(ref.mx8_half_steps(torch.from_numpy(scales), 34)[0, [0, 33]], [0.5, 1.0])


@pytest.mark.parametrize("a", range(5))
def test_reference_slopes(a):
    """The derivatives against central differences."""
    v = torch.linspace(-6.0, 6.0, 240).double() + 1e-3
    h = 1e-6
    d = (ref.act(v + h, a) - ref.act(v - h, a)) / (2 * h)
    assert float((d - ref.slope(v, a)).abs().max()) < 1e-8


@pytest.mark.parametrize("scoring", range(4))
def test_reference_router_gradient(scoring):
    """The formulas against the graph's derivative of the same loss and weights."""
    g = torch.Generator().manual_seed(scoring)
    T, E, k = 7, 9, 3
    logits = torch.randn(T, E, generator=g).double().requires_grad_(True)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32)
    dw = torch.randn(T, k, generator=g)
    loss, counts, slopes = ref.balance(logits, ids, scoring)
    p = torch.softmax(logits, -1) if scoring < 2 else torch.sigmoid(logits) / torch.sigmoid(logits).sum(-1, keepdim=True)
    f = counts.double() / (T * k)
    own = E * (f * p.mean(0)).sum()
    assert abs(float(own.detach()) - float(loss.detach())) < 1e-12
    ix = ids.long()
    w = {0: lambda: p.gather(1, ix), 1: lambda: torch.softmax(logits.gather(1, ix), -1),
         2: lambda: torch.sigmoid(logits.gather(1, ix)),
         3: lambda: torch.sigmoid(logits.gather(1, ix)) / torch.sigmoid(logits.gather(1, ix)).sum(-1, keepdim=True)}[scoring]()
    (2.0 * own + (w * dw.double()).sum()).backward()
    d, _ = ref.route_backward(logits, ids, dw, slopes, 2.0, scoring)
    assert float((d - logits.grad).abs().max()) < 1e-12
