"""The products with 16-bit weights, the bias's gradient and the router's loss and gradient through the LDS-poison debug
build (every kernel fills its LDS with NaN bits or large integers before it uses it): the same bits as from the product
build, on every kernel and tile shape."""
import os

import pytest
import torch

import quantized_swiglu_forward_amd as swq
from gpu_helpers import say
from test_gpu_dense import BF16, F16, F32, normal
from test_gpu_train import choice

pytestmark = pytest.mark.gpu

POISON = os.path.join(os.path.dirname(swq.LIB_PATH), "libswiglu_q_ldspoison.so")


@pytest.fixture(scope="module")
def poison():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    assert os.path.exists(POISON), f"{POISON} is not built"
    yield swq.load_library(POISON)
    torch.cuda.synchronize()


def both(poison, run):
    product = swq.lib()
    want = run()
    swq._lib = poison
    try:
        got = run()
        torch.cuda.synchronize()
    finally:
        swq._lib = product
    for a, b in zip(got, want):
        assert torch.equal(a, b) and not (a.is_floating_point() and torch.isnan(a).any())


# few rows (one, two and four row tiles, one and two column tiles), tiles of 64, 128, 256 and 256 x 192, splits
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("M,K,N", [(1, 544, 33), (1, 2048, 5632), (20, 288, 500), (50, 161, 96), (40, 2080, 4100), (70, 200, 1030),
                                   (300, 4096, 128), (1100, 160, 2400), (2100, 96, 5600), (3000, 96, 4200)])
def test_layer(poison, M, K, N, dtype):
    x, w, bias = normal(M, M, K, dtype=dtype), normal(N, N, K, dtype=dtype, scale=K ** -0.5), normal(2, N, dtype=dtype)
    dout = normal(3, M, N, dtype=dtype)
    say("poison dense", M, K, N, dtype)

    def run():
        y, z = swq.dense_linear(x, w, bias, act=swq.SWQ_ACT_GELU, keep="mx8")
        plain = swq.dense_linear(x, w, residual=dout, out_mode=swq.SWQ_LINEAR_F32)
        return (y, *z, plain, *swq.dense_linear_backward(dout, swq.mx8_quantize(x), w, z, act=swq.SWQ_ACT_GELU),
                swq.dense_linear_backward(dout, None, w, want=(False, False, True))[2])

    both(poison, run)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("T,E,k", [(1, 8, 2), (100, 64, 20), (1000, 100, 8), (700, 256, 30), (300, 500, 10), (400, 1024, 64)])
def test_router(poison, T, E, k, dtype):
    logits, dw = choice(T, E, k, dtype)
    say("poison router", T, E, k, dtype)
    for scoring in (swq.SWQ_ROUTE_SOFTMAX, swq.SWQ_ROUTE_SIGMOID_CHOSEN):
        def run():
            ids, _ = swq.route(logits, k, scoring)
            loss, counts, slopes = swq.balance_loss(logits, ids, scoring)
            return loss, counts, slopes, swq.route_backward(logits, ids, dw, scoring, slopes=slopes)

        both(poison, run)
