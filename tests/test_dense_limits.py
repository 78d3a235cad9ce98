"""Sizes at the ends of what the products with 16-bit weights take, and the bounds of a checkpoint's values, without a GPU."""
import pytest
import torch

import dense_reference as ref
import quantized_swiglu_forward_amd as swq

P = 1 << 20    # a fake, aligned "device" address: validation never dereferences it
LINEAR = dict(x=P, W=P, bias=P, residual=P, M=4, K=16, N=64, type=0, act=2, out_mode=0, out=P, stream=0)
BACK = dict(dout=P, x=P, x_scales=None, W=P, z=None, z_scales=None, M=4, K=16, N=64, type=0, act=0, dx=P, dW=P, dbias=P,
            stream=0)
MOST = 1 << 30


@pytest.mark.parametrize("fn,base,kw", [
    (swq.swiglu_q_dense_linear, LINEAR, dict(M=MOST, N=512)),                 # 2^23 tiles of 512 threads
    (swq.swiglu_q_dense_linear, LINEAR, dict(M=MOST, N=1 << 20)),
    (swq.swiglu_q_dense_linear_backward, BACK, dict(M=MOST, K=512)),
    (swq.swiglu_q_dense_linear_backward, BACK, dict(M=MOST, K=512, dW=None, dbias=None)),
    (swq.swiglu_q_dense_linear_backward, BACK, dict(M=64, K=1 << 20, N=1 << 20, dx=None)),
])
def test_more_threads_than_a_launch(fn, base, kw):
    """A launch of 2^32 threads or more would be cut off without an error: such a product is refused."""
    assert fn(**{**base, **kw}) == swq.SWQ_ERR_SHAPE


@pytest.mark.parametrize("fn,base,kw", [
    (swq.swiglu_q_dense_linear, LINEAR, dict(M=MOST, N=1)),
    (swq.swiglu_q_dense_linear, LINEAR, dict(M=MOST, N=64)),
    (swq.swiglu_q_dense_linear, LINEAR, dict(M=MOST, N=256)),
    (swq.swiglu_q_dense_linear, LINEAR, dict(M=1 << 17, N=1 << 20)),
    (swq.swiglu_q_dense_linear_backward, BACK, dict(M=MOST, N=8)),
    (swq.swiglu_q_dense_linear_backward, BACK, dict(M=MOST, N=8, K=256)),
    (swq.swiglu_q_dense_linear_backward, BACK, dict(M=8, K=1 << 18, N=1 << 18)),
])
def test_sizes_that_are_taken(fn, base, kw):
    """What the card's memory could hold is not refused: without a GPU the call fails only where it needs one."""
    if torch.cuda.is_available():
        pytest.skip("would launch on addresses that are none")
    assert fn(**{**base, **kw}) in (swq.SWQ_ERR_HIP, swq.SWQ_ERR_WORKSPACE)


def test_operands_that_are_not_read():
    """x without dW may lie at any address, with it it may not (no rows and no dW: nothing to launch); likewise W without dx."""
    none = dict(M=0, dW=None, dbias=None)
    assert swq.swiglu_q_dense_linear_backward(**{**BACK, **none, "x": P + 2}) == swq.SWQ_OK
    assert swq.swiglu_q_dense_linear_backward(**{**BACK, **none, "W": P + 2}) == swq.SWQ_ERR_ALIGN
    assert swq.swiglu_q_dense_linear_backward(**{**BACK, "x": P + 2, "dx": None}) == swq.SWQ_ERR_ALIGN
    assert swq.swiglu_q_dense_linear_backward(**{**BACK, "x": P + 2}) == swq.SWQ_ERR_ALIGN
    assert swq.swiglu_q_dense_linear_backward(**{**BACK, "W": P + 2}) == swq.SWQ_ERR_ALIGN


@pytest.mark.parametrize("low,high", [(-149, -127), (-126, -121), (-120, -118), (-3, 3), (125, 128)])
def test_how_far_a_checkpoint_is_off(low, high):
    """The documented bounds, over float32's whole range: half a step, 1/127 of the block's largest magnitude from 2^-120 on, a
    whole step from 127.5 2^121 on.  (The GPU's codes and scales are these, bit by bit, in the tests of the checkpoints.)"""
    g = torch.Generator().manual_seed(high)
    # (one rounding, to float32, where this is the checkpoint's input)
    x = (torch.rand(60, 64, generator=g).double() * torch.exp2(torch.randint(low, high + 1, (60, 1), generator=g).double()))
    x = (x * torch.where(torch.rand(60, 64, generator=g) < 0.5, -1.0, 1.0)).clamp(max=torch.finfo(torch.float32).max).float()
    x[0, 0] = torch.finfo(torch.float32).max if high == 128 else 2.0 ** low
    codes, scales = (torch.from_numpy(t) for t in ref.mx8(x))
    off = (ref.mx8_values(codes, scales) - x.double()).abs()
    half = ref.mx8_half_steps(scales, 64)
    top = x.double().abs().view(60, 2, 32).amax(-1).repeat_interleave(32, -1)
    last = x.double().abs() >= 127.5 * 2.0 ** 121
    assert bool((off <= torch.where(last, 2 * half, half)).all()) and bool((scales >= 7).all()) and bool((scales <= 254).all())
    assert bool((off <= top / 127)[top >= 2.0 ** -120].all())
    # both exceptions are there (values are 2^low times a factor below 1, so with low = -120 some blocks lie under the border; a
    # whole step of 127.5 and more is under 1/127 of them)
    assert bool((off > half).any()) == (high == 128) and bool((off > top / 127).any()) == (low <= -120)
