"""Sizes at the ends of what the MXFP4 operators, the router and the experts'
MLP take, without a GPU: what they refuse, they refuse before any HIP call."""
import pytest
import torch

import quantized_swiglu_forward_amd as swq


def mx(*shape):
    return torch.zeros(*shape[:-1], shape[-1] // 8, dtype=torch.int32), torch.zeros(*shape[:-1], shape[-1] // 32,
                                                                                     dtype=torch.uint8)


def rows(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


CHOSEN = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)


@pytest.mark.parametrize("call", [
    lambda: swq.mx4_linear(rows(4, 0), *mx(8, 0)),
    lambda: swq.mx4_linear(rows(4, 0), *mx(8, 0), residual=rows(4, 8)),
    lambda: swq.mx4_matmul(*mx(4, 0), *mx(8, 0)),
    lambda: swq.mx4_grouped_linear(rows(4, 0), torch.zeros(4, dtype=torch.int32), *mx(3, 8, 0)),
    lambda: swq.moe_mlp(rows(4, 0), *CHOSEN, *mx(3, 32, 0), *mx(3, 32, 0), *mx(3, 64, 32), residual=rows(4, 64)),
    lambda: swq.moe_mlp(rows(4, 64), *CHOSEN, *mx(3, 0, 64), *mx(3, 0, 64), *mx(3, 64, 0)),
])
@pytest.mark.parametrize("anywhere", [False, True], ids=["cpu", "as-on-gpu"])
def test_no_inputs(call, anywhere, monkeypatch):
    """A product over no inputs is refused: nothing would write its output."""
    if anywhere:        # as if the tensors were on a GPU; nothing may reach the library
        monkeypatch.setattr(swq, "_same_place", lambda what, x, *tensors: 0)
        monkeypatch.setattr(swq, "_call", lambda *a: pytest.fail("launched"))
    with pytest.raises(ValueError, match="K = 0"):
        call()


P = 1 << 20    # a fake, aligned "device" address: validation never dereferences it
LINEAR = dict(x=P, W=P, s=P, residual=None, M=4, K=32, N=8, type=0, out_mode=0, out=P, stream=0)
GROUPED = dict(x=P, offsets=P, W=P, s=P, P=4, E=3, K=32, N=8, type=0, out_mode=0, out=P, stream=0)
MOE = dict(x=P, ids=P, weights=P, Wg=P, sg=P, Wu=P, su=P, Wd=P, sd=P, residual=None, T=4, k=2, E=8, H=32, I=32, Ho=64,
           type=0, out_mode=0, out=P, stream=0)


@pytest.mark.parametrize("fn,base,kw", [
    (swq.swiglu_q_mx4_linear, LINEAR, dict(M=1, N=1 << 28)),                  # 16 columns a block of 256 threads
    (swq.swiglu_q_mx4_linear, LINEAR, dict(M=1, K=4096, N=1 << 27)),          # ... of 512
    (swq.swiglu_q_mx4_linear, LINEAR, dict(M=2, N=1 << 30)),                  # 64 columns a block of 512
    (swq.swiglu_q_mx4_linear, LINEAR, dict(M=2, N=1 << 30, type=2, out_mode=2)),
    (swq.swiglu_q_mx4_linear, LINEAR, dict(M=1 << 30, N=8, type=2, out_mode=2)),      # 64 rows a block of 256
    (swq.swiglu_q_mx4_grouped_linear, GROUPED, dict(P=4096, E=1024, N=1 << 20)),
    (swq.swiglu_q_moe_mlp, MOE, dict(T=1, k=2, Ho=1 << 26)),                  # slot by slot: outputs
    (swq.swiglu_q_moe_mlp, MOE, dict(T=64, k=64, E=1024, I=1 << 20)),         # by expert
])
def test_more_threads_than_a_launch(fn, base, kw):
    """A launch of 2^32 threads or more would be cut off without an error: such a product is refused."""
    assert fn(**{**base, **kw}) == swq.SWQ_ERR_SHAPE
