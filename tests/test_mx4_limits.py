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
