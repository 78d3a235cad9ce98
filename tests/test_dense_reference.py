"""The bounds that the GPU tests of the products with 16-bit weights, the checkpoints and the router's gradient use
(dense_reference): a float32 computation with the documented roundings passes, planted mistakes do not (CPU)."""
import pytest
import torch

import dense_reference as ref

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def gen(seed, *shape, dtype=BF16, scale=1.0):
    return (scale * torch.randn(*shape, generator=torch.Generator().manual_seed(seed))).to(dtype)


def layer(dtype, M=9, K=70, N=41):
    return gen(1, M, K, dtype=dtype), gen(2, N, K, dtype=dtype, scale=K ** -0.5), gen(3, N, dtype=dtype), gen(4, M, N, dtype=dtype)


def act32(z, a):
    s = torch.sigmoid
    return (z, z.clamp(min=0), z * s(z), 0.5 * z * (1 + torch.erf(z * 2 ** -0.5)),
            z * s(1.5957691 * (z + 0.044715 * z ** 3)))[a]


FORWARD = {
    "none": lambda x, w, b, r: (x, w, b, r),
    "last inner index": lambda x, w, b, r: (torch.cat([x[:, :-1], 0 * x[:, -1:]], 1), w, b, r),
    "last inner index twice": lambda x, w, b, r: (torch.cat([x[:, :-1], 2 * x[:, -1:]], 1), w, b, r),
    "bias of one column": lambda x, w, b, r: (x, w, torch.cat([b[:-1], 0 * b[-1:]]), r),
    "residual of the row before": lambda x, w, b, r: (x, w, b, r.roll(1, 0)),
    "one weight": lambda x, w, b, r: (x, torch.cat([w[:7], w[7:8].roll(1, 1), w[8:]]), b, r),
}


@pytest.mark.parametrize("mistake", FORWARD)
@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (F16, F16), (BF16, F32), (F16, F32)])
@pytest.mark.parametrize("a", range(5))
def test_forward(mistake, dtype, out, a):
    x, w, b, r = layer(dtype)
    want, z, err = ref.linear(x, w, b, r, a)
    mx, mw, mb, mr = FORWARD[mistake](x, w, b, r)
    got = (act32(mx.float() @ mw.float().t() + mb.float(), a) + mr.float()).to(out)
    check = lambda: ref.close(got, want, ref.linear_tol(z, err, r, a, want, out), mistake)  # noqa: E731
    if mistake == "none":
        check()
    else:
        with pytest.raises(AssertionError):
            check()


@pytest.mark.parametrize("a,b", [(3, 4), (4, 3), (2, 3), (1, 3), (0, 1)])
def test_another_activation(a, b):
    x, w, bias, r = layer(F16)
    want, z, err = ref.linear(x, w, bias, None, a)
    got = act32(x.float() @ w.float().t() + bias.float(), b)
    with pytest.raises(AssertionError):
        ref.close(got, want, ref.linear_tol(z, err, None, a, want, F32))


BACKWARD = {
    "none": lambda d, s, x, w: (d * s, x, w),
    "slope of the next column": lambda d, s, x, w: (d * s.roll(1, 1), x, w),
    "last row": lambda d, s, x, w: (torch.cat([(d * s)[:-1], 0 * d[-1:]]), x, w),
    "last column": lambda d, s, x, w: (torch.cat([(d * s)[:, :-1], 0 * d[:, -1:]], 1), x, w),
    "no slope": lambda d, s, x, w: (d, x, w),
}


@pytest.mark.parametrize("mistake", BACKWARD)
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("a", range(1, 5))
def test_backward(mistake, dtype, a):
    x, w, b, dout = layer(dtype)
    z = (x.float() @ w.float().t() + b.float()).to(dtype)
    want = ref.backward(dout, ref.wide(x), w, ref.wide(z), a, dtype)
    dz, mx, mw = BACKWARD[mistake](dout.float(), ref.slope(ref.wide(z), a).float(), x, w)
    d16 = dz.to(dtype).float()
    got = {"dx": (d16 @ mw.float()).to(dtype), "dw": (d16.t() @ mx.float()).to(dtype), "dbias": dz.sum(0).to(dtype)}
    wrong = 0
    for name, (v, tol) in want.items():
        if mistake == "none":
            ref.close(got[name], v, tol, name)
        else:
            try:
                ref.close(got[name], v, tol, name)
            except AssertionError:
                wrong += 1
    assert wrong == (0 if mistake == "none" else 3)


@pytest.mark.parametrize("mistake", ["none", "scale", "row", "truncated"])
def test_checkpoint_of_sums(mistake):
    """A checkpoint made from float32 sums: the codes of the 64-bit ones up to half a step."""
    x, w, b, _ = layer(BF16, N=64)
    z32 = x.float() @ w.float().t() + b.float()
    _, z, err = ref.linear(x, w, b, None, 0)
    codes, scales = (torch.from_numpy(t) for t in ref.mx8(z32))
    if mistake == "scale":
        scales[4, 1] += 1
    elif mistake == "row":
        codes[3] = codes[2]
    elif mistake == "truncated":
        steps = torch.ldexp(torch.ones(()).double(), scales - 133).repeat_interleave(32, -1)
        codes = torch.trunc(ref.wide(z32) / steps)
    check = lambda: ref.close(ref.mx8_values(codes, scales), z, err + ref.mx8_half_steps(scales, 64) * 1.01)  # noqa: E731
    if mistake == "none":
        check()
    else:
        with pytest.raises(AssertionError):
            check()


ROUTER = ["none", "duplicates once", "tokens without a slot", "no second factor", "softmax over all"]


@pytest.mark.parametrize("mistake", ROUTER)
def test_router(mistake):
    """Slots twice, ids outside the experts, tokens without a slot."""
    T, E, k, scoring = 30, 9, 4, 3
    logits, dw = gen(1, T, E, dtype=F32, scale=2.0), gen(2, T, k, dtype=F32)
    ids = torch.randint(-2, E + 2, (T, k), generator=torch.Generator().manual_seed(3)).to(torch.int32)
    ids[4] = torch.tensor([2, 2, 3, 5])      # (four times the same would have no gradient, once or four times)
    ids[5] = -1
    loss, counts, slopes = ref.balance(logits, ids, scoring)
    want, tol = ref.route_backward(logits, ids, dw, slopes, 1.0, scoring)
    got = want.float()
    if mistake == "duplicates once":
        once = ids.clone()
        once[4, 1] = -1
        got = ref.route_backward(logits, once, dw, slopes, 1.0, scoring)[0]
    elif mistake == "tokens without a slot":
        live = torch.zeros_like(ids)
        p = ref.shares(logits.double(), scoring)
        got = want + torch.where((live == ids[5]).all(-1, keepdim=True), p, 1e-3 * p)
    elif mistake == "no second factor":
        got = want / torch.sigmoid(-logits.double())
    elif mistake == "softmax over all":
        got = ref.route_backward(logits, ids, dw, slopes, 1.0, 0)[0]
    if mistake == "none":
        ref.close(got, want, tol + ref.rounding(want, F32))
    else:
        with pytest.raises(AssertionError):
            ref.close(got, want, tol + ref.rounding(want, F32))
    share = ref.balance(logits, torch.where(ids < 0, torch.zeros_like(ids), ids), scoring)
    assert not torch.equal(share[1], counts) and abs(float(share[0] - loss)) > 1e-3
