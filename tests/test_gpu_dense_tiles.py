"""The dense products at sizes that take the larger tiles (128 x 128, 256 x 256, 256 x 192 forward, 128 and 256 for the
gradients, with and without splits of the inner index): rows and columns at the tiles' borders against 64 bits, every
element against float32 sums."""
import pytest
import torch

import dense_reference as ref
import quantized_swiglu_forward_amd as swq
from gpu_helpers import say
from test_gpu_dense import BF16, F16, F32, MODE, layer, normal

pytestmark = pytest.mark.gpu

# 128 x 128 twice, 256 x 256 twice, 256 x 192 twice: inner sizes below, at and past whole steps, odd and whole rows
FORWARD = [(1283, 72, 1537), (1291, 201, 1541), (3001, 136, 4104), (3001, 331, 4099), (1537, 40, 5125), (1540, 330, 5120)]
# 128 x 128 plain, dW's rows split, dx's columns split, both split; 256 x 256
BACKWARD = [(700, 2050, 700), (8200, 330, 385), (385, 330, 8200), (5125, 65, 6150), (1537, 4099, 4099)]


def some(n):
    """Indexes below n around the tiles' borders, and a few others."""
    at = {0, n - 1, n - 2, n // 2, n // 3}
    for step in (64, 128, 192, 256):
        last = (n - 1) // step * step
        at |= {step - 1, step, last - 1, last}
    return torch.tensor(sorted(i for i in at if 0 <= i < n))


def whole(got, a, b, dtype, what):
    """Every element of a b^T in dtype against float32 sums of float32 products: either side off by the sums' bound."""
    a, b = a.float(), b.float()
    want, mass = torch.matmul(a, b.t()), torch.matmul(a.abs(), b.abs().t())
    off = (got.float() - want).abs() - 2 * (a.shape[1] + 2) * ref.SUM * mass - 1.01 * ref.U[dtype] * want.abs()
    assert float(off.max()) <= (2.0 ** -24 if dtype == F16 else 0.0), f"{what}: off by {float(off.max()):.3g} too much"


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("M,K,N", FORWARD)
def test_forward(M, K, N, dtype):
    x, w, bias, residual = layer(M, K, N, dtype)
    rows = some(M)
    sub, at = x.cpu()[rows], rows.cuda()
    for act, b, r, keep, out in ((0, None, None, None, F32), (3, bias, residual, None, dtype), (2, bias, residual, "mx8", dtype),
                                 (4, None, residual, "same", F32), (1, bias, None, "mx8", F32)):
        say("dense tiles", M, K, N, dtype, act, keep)
        got = swq.dense_linear(x, w, b, act=act, residual=r, keep=keep, out_mode=MODE[out])
        y, z = got if keep else (got, None)
        res = None if r is None else r[at]
        want, wz, err = ref.linear(sub, w, b, res, act)
        ref.close(y[at], want, ref.linear_tol(wz, err, res, act, want, out), f"out, act {act}")
        if keep == "same":
            ref.close(z[at], wz, err + ref.rounding(wz, dtype) * 1.01, "z")
            whole(z, x, w, dtype, "z")
        elif keep == "mx8":
            code, scale = z[0][at], z[1][at]
            ref.close(ref.mx8_values(code, scale), wz, err + ref.mx8_half_steps(scale, N) * 1.01, "checkpoint of z")
        elif act == 0:
            whole(y, x, w, F32, "out")


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("M,K,N", BACKWARD)
def test_backward(M, K, N, dtype):
    x, w, bias, _ = layer(M, K, N, dtype)
    dout = normal(M * 3 + N, M, N, dtype=dtype)
    rows, columns = some(M), some(N)
    say("dense tiles, backward", M, K, N, dtype)
    dx, dw, _ = swq.dense_linear_backward(dout, x, w)
    whole(dx, dout, w.t().contiguous(), dtype, "dx")
    whole(dw, dout.t().contiguous(), x.t().contiguous(), dtype, "dw")
    x8 = swq.mx8_quantize(x)
    _, z = swq.dense_linear(x, w, bias, act=2, keep="mx8")
    say("dense tiles, backward with checkpoints", M, K, N, dtype)
    dx, dw, db = swq.dense_linear_backward(dout, x8, w, z, act=2)
    wx, wz = ref.mx8_values(*x8), ref.mx8_values(*z)
    if dtype == F16:                                           # decoded to binary16 for the product
        wx = wx.to(F16).double()
    d = dout.cpu()
    want, tol = ref.backward(d[rows], wx[rows], w, wz[rows], 2, dtype)["dx"]
    ref.close(dx[rows.cuda()], want, tol, "dx")
    at = columns.cuda()
    part = ref.backward(d[:, columns], wx, w[at], wz[:, columns], 2, dtype)
    ref.close(dw[at], *part["dw"], "dw")
    ref.close(db[at], *part["dbias"], "dbias")
