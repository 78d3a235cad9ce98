"""The MXFP4 operators and the experts' MLP through the LDS-poison debug build
(every kernel fills its LDS with NaN bits before it uses it): the same bits as
from the product build, on every kernel and tile shape."""
import os

import pytest
import torch

import quantized_swiglu_forward_amd as swq
from gpu_helpers import say
from test_gpu_mx4 import BF16, F16, acts, matrix, moe_case

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
    assert torch.equal(got, want) and not torch.isnan(got).any()


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("M,K,N", [(1, 4160, 130), (1, 544, 33), (7, 1056, 300), (20, 288, 9000), (24, 96, 70),
                                   (40, 2080, 300), (200, 160, 4096), (600, 96, 5632), (1900, 96, 4096)])
def test_linear(poison, M, K, N, dtype):
    x, (w, s) = acts(M, M, K, dtype=dtype), matrix(N, N, K)
    say("poison mx4 linear", M, K, N, dtype)
    both(poison, lambda: swq.mx4_linear(x, w, s))


@pytest.mark.parametrize("M,K,N", [(3, 1056, 70), (40, 160, 300), (500, 544, 1030), (1500, 160, 1530), (3100, 288, 3336)])
def test_matmul(poison, M, K, N):
    (a, sa), (w, s) = matrix(M, M, K), matrix(N, N, K)
    say("poison mx4 matmul", M, K, N)
    both(poison, lambda: swq.mx4_matmul(a, sa, w, s))


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("P,E", [(20, 5), (45, 3), (300, 4), (2600, 3)])
def test_grouped(poison, P, E, dtype):
    x, (w, s) = acts(P, P, 352, dtype=dtype), matrix(E, E, 260, 352)
    off = torch.linspace(0, P, E + 1).to(torch.int32).cuda()
    say("poison grouped", P, E, dtype)
    both(poison, lambda: swq.mx4_grouped_linear(x, off, w, s))


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("T,k,E,H,I", [(1, 4, 8, 2080, 1056), (3, 2, 4, 96, 64), (20, 2, 8, 96, 64), (300, 3, 5, 96, 288),
                                       (900, 2, 3, 64, 4096)])
def test_moe(poison, T, k, E, H, I, dtype):
    x, ids, weights, ((wg, sg), (wu, su), (wd, sd)) = moe_case(T, T, k, E, H, I, 130, dtype)
    say("poison moe", T, k, E, H, I, dtype)
    both(poison, lambda: swq.moe_mlp(x, ids, weights, wg, sg, wu, su, wd, sd))
