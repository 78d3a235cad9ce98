"""More mistakes planted in the reference forms of the router's loss and gradient (dense_reference): each leaves the bounds that
the GPU tests use, and nothing else does (CPU)."""
import pytest
import torch

import dense_reference as ref

F32 = torch.float32


def gen(seed, *shape, scale=1.0):
    return scale * torch.randn(*shape, generator=torch.Generator().manual_seed(seed))


def fails(got, want, tol):
    with pytest.raises(AssertionError):
        ref.close(got, want, tol)


@pytest.mark.parametrize("scoring", range(4))
def test_a_token_without_a_slot(scoring):
    """The balance loss's gradient given to a token that has no slot, every other row left as it is."""
    T, E, k, bare = 30, 9, 4, 5
    logits, dw = gen(1, T, E, scale=2.0), gen(2, T, k)
    ids = torch.randint(0, E, (T, k), generator=torch.Generator().manual_seed(3)).to(torch.int32)
    ids[bare] = torch.tensor([-1, E, -7, E + 3])
    _, _, slopes = ref.balance(logits, ids, scoring)
    want, tol = ref.route_backward(logits, ids, dw, slopes, 1.0, scoring)
    tol = tol + ref.rounding(want, F32)
    v = logits[bare].double()
    p = ref.shares(v[None], scoring)[0]
    g = p * (slopes - (slopes * p).sum())
    if scoring >= 2:
        g = g * torch.sigmoid(-v)
    got = want.clone()
    got[bare] += g
    assert bool((g != 0).any()) and not want[bare].any()
    fails(got, want, tol)
    rest = torch.arange(T) != bare
    ref.close(got[rest], want[rest], tol[rest])
    ref.close(want.float(), want, tol)


@pytest.mark.parametrize("scoring", range(4))
def test_a_masked_expert_in_a_slot(scoring):
    """A slot whose expert is masked: its dweights entry changes nothing.  Taken with the weight of a logit of 0, it does."""
    T, E, k = 6, 7, 3
    logits, dw = gen(4, T, E), gen(5, T, k)
    ids = torch.tensor([[0, 1, 2]] * T, dtype=torch.int32)
    logits[:, 1] = float("-inf")
    want, tol = ref.route_backward(logits, ids, dw, None, 1.0, scoring)
    tol = tol + ref.rounding(want, F32)
    other = dw.clone()
    other[:, 1] = 100.0
    ref.close(ref.route_backward(logits, ids, other, None, 1.0, scoring)[0], want, tol)
    seen = torch.where(torch.isinf(logits), torch.zeros_like(logits), logits)
    fails(ref.route_backward(seen, ids, other, None, 1.0, scoring)[0], want, tol)


@pytest.mark.parametrize("a", [2, 3])
@pytest.mark.parametrize("side", [1.0, -1.0])
def test_a_derivative_at_infinity(a, side):
    """An infinite z times a factor of 0 is NaN where the derivative is 1 or 0."""
    z = torch.tensor([[side * 72000.0, 0.5]]).double()
    want = ref.backward(torch.ones(1, 2), torch.ones(1, 1).double(), torch.ones(2, 1), z, a, torch.float16)["dbias"]
    assert want[0][0] == max(side, 0.0)
    ref.close(want[0].float(), *want)
    got = want[0].clone()
    got[0] = float("nan")
    fails(got, *want)
