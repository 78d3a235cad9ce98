"""The products with 16-bit weights and their gradients on the GPU against
their plain 64-bit forms (dense_reference), within the bounds derived there."""
import pytest
import torch

import dense_reference as ref
import quantized_swiglu_forward_amd as swq
from gpu_helpers import say

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
MODE = {BF16: swq.SWQ_LINEAR_BF16, F16: swq.SWQ_LINEAR_F16, F32: swq.SWQ_LINEAR_F32}


@pytest.fixture(autouse=True, scope="module")
def _device():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    swq.lib()
    yield
    torch.cuda.synchronize()


def normal(seed, *shape, dtype=BF16, scale=1.0):
    return (scale * torch.randn(*shape, generator=torch.Generator().manual_seed(seed))).to(dtype).cuda()


def layer(M, K, N, dtype):
    return (normal(M + 1, M, K, dtype=dtype), normal(K + 2, N, K, dtype=dtype, scale=2 * K ** -0.5),
            normal(N + 3, N, dtype=dtype), normal(M + N, M, N, dtype=dtype))


def check_forward(x, w, bias, residual, act, out_dtype, keep, what):
    M = x.shape[0]
    got = swq.dense_linear(x, w, bias, act=act, residual=residual, keep=keep, out_mode=MODE[out_dtype])
    y, z = got if keep else (got, None)
    want, wz, err = ref.linear(x, w, bias, residual, act)
    ref.close(y, want, ref.linear_tol(wz, err, residual, act, want, out_dtype), f"{what} out")
    if keep == "same":
        ref.close(z, wz, err + ref.rounding(wz, x.dtype) * 1.01, f"{what} z")
    elif keep == "mx8":
        v, half = ref.mx8_values(*z), ref.mx8_half_steps(z[1], w.shape[0])
        ref.close(v, wz, err + half * 1.01, f"{what} checkpoint of z")
        # the step is the smallest: the largest code of a block is above 63
        top = torch.nn.functional.pad(z[0].int().abs(), (0, -w.shape[0] % 32)).reshape(M, -1, 32).amax(-1)
        assert bool((top >= 63).all()), f"{what}: a coarser step than needed"
    return y, z


SIZES = [(1, 1, 1), (1, 7, 5), (1, 2048, 300), (2, 96, 17), (3, 4099, 33), (5, 31, 129), (7, 1000, 64), (16, 512, 100),
         (17, 1056, 257), (31, 64, 2049), (33, 65, 130), (40, 2080, 513), (64, 1024, 515), (65, 353, 128),
         (100, 2048, 31), (127, 33, 640), (129, 256, 641), (200, 992, 1001), (257, 1537, 259), (300, 130, 1300),
         (520, 72, 770), (700, 640, 1025)]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("M,K,N", SIZES)
def test_forward(M, K, N, dtype):
    x, w, bias, residual = layer(M, K, N, dtype)
    say("dense linear", M, K, N, dtype)
    check_forward(x, w, None, None, 0, F32, None, "plain")
    check_forward(x, w, bias, residual, swq.SWQ_ACT_GELU, dtype, None, "epilogue")
    check_forward(x, w, bias, None, swq.SWQ_ACT_SILU, dtype, "mx8", "mx8")
    check_forward(x, w, None, residual, swq.SWQ_ACT_GELU_TANH, F32, "same", "same")


@pytest.mark.parametrize("act", range(5))
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("M,K,N", [(3, 64, 72), (150, 40, 99), (600, 64, 800)])
def test_activations(M, K, N, dtype, act):
    """Values of both signs, small and far from zero."""
    x, w, bias, residual = layer(M, K, N, dtype)
    x = x * torch.logspace(-2, 1, M, device="cuda")[:, None].to(dtype)
    say("activation", M, K, N, dtype, act)
    for keep in (None, "same", "mx8"):
        check_forward(x, w, bias, residual, act, F32, keep, f"act {act} {keep}")


@pytest.mark.parametrize("keep", ["same", "mx8"])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("M,K,N", [s for s in SIZES])
def test_backward(M, K, N, dtype, keep):
    x, w, bias, _ = layer(M, K, N, dtype)
    act = (swq.SWQ_ACT_GELU, swq.SWQ_ACT_SILU, swq.SWQ_ACT_GELU_TANH, swq.SWQ_ACT_RELU)[(M + N) % 4]
    dout = normal(M * 3 + N, M, N, dtype=dtype)
    say("dense backward", M, K, N, dtype, keep, act)
    _, z = swq.dense_linear(x, w, bias, act=act, keep=keep)
    kept, wx, wz = x, ref.wide(x), None
    if keep == "mx8":
        kept = swq.mx8_quantize(x)
        wx, wz = ref.mx8_values(*kept), ref.mx8_values(*z)
        if dtype == F16:                                       # decoded to binary16 for the product
            wx = wx.to(F16).double()
    else:
        wz = ref.wide(z)
    got = dict(zip(("dx", "dw", "dbias"), swq.dense_linear_backward(dout, kept, w, z, act=act)))
    for name, (want, tol) in ref.backward(dout, wx, w, wz, act, dtype).items():
        ref.close(got[name], want, tol, name)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("M,K,N", [(1, 40, 24), (9, 33, 65), (130, 128, 264), (513, 260, 96)])
def test_backward_without_activation(M, K, N, dtype):
    x, w, _, _ = layer(M, K, N, dtype)
    dout = normal(M * 5 + N, M, N, dtype=dtype)
    say("dense backward, no activation", M, K, N, dtype)
    got = dict(zip(("dx", "dw", "dbias"), swq.dense_linear_backward(dout, x, w)))
    want = ref.backward(dout, ref.wide(x), w, None, 0, dtype)
    for name, (v, tol) in want.items():
        ref.close(got[name], v, tol, name)
    for i, name in enumerate(("dx", "dw", "dbias")):           # each alone gives the same bits
        alone = swq.dense_linear_backward(dout, x, w, want=[j == i for j in range(3)])
        assert torch.equal(alone[i], got[name]) and all(alone[j] is None for j in range(3) if j != i)


@pytest.mark.parametrize("act", range(1, 5))
def test_gradient_against_differences(act):
    """dx, dw and dbias against central differences of the 64-bit forward form.  The differences' own error, h^2 / 6 of
    the third derivative plus 2^-52 / h, is below 1e-7 of the terms at h = 1e-4 (RELU has its kinks
    away from the points taken); what counts is the outputs' and dz's rounding to 16 bits."""
    M, K, N, dtype = 4, 6, 5, F16
    x, w, bias, _ = layer(M, K, N, dtype)
    dout = normal(9, M, N, dtype=dtype)
    say("differences", act)
    _, z = swq.dense_linear(x, w, bias, act=act, keep="same")
    got = dict(zip(("dx", "dw", "dbias"), swq.dense_linear_backward(dout, x, w, z, act=act)))
    args = {"dx": ref.wide(x), "dw": ref.wide(w), "dbias": ref.wide(bias)}

    def value(a):
        zz = a["dx"] @ a["dw"].t() + a["dbias"]
        return float((ref.act(zz, act) * ref.wide(dout)).sum())

    zz = ref.wide(x) @ ref.wide(w).t() + ref.wide(bias)
    assert act != swq.SWQ_ACT_RELU or float(zz.abs().min()) > 2e-3
    # z's own rounding to binary16 moves act' by at most 1.2 |z| 2^-11 (|act''| < 1.2)
    tols = ref.backward(dout, ref.wide(x), w, ref.wide(z), act, dtype)
    zoff = ref.wide(dout).abs() * (1.2 * zz.abs() * 2.0 ** -11 + 2.0 ** -24 if act > 1 else 0.0 * zz)
    more = {"dx": zoff @ ref.wide(w).abs(), "dw": zoff.t() @ ref.wide(x).abs(), "dbias": zoff.sum(0)}
    h = 1e-4
    for name, at in args.items():
        d = torch.zeros_like(at)
        for i in range(at.numel()):
            for sign in (1, -1):
                moved = at.clone().reshape(-1)
                moved[i] += sign * h
                d.view(-1)[i] += sign * value({**args, name: moved.reshape(at.shape)}) / (2 * h)
        ref.close(got[name], d, tols[name][1] + more[name] + 1e-6, name)


def test_no_rows():
    w = normal(1, 24, 40)
    say("no rows")
    x, dout = torch.empty(0, 40, dtype=BF16, device="cuda"), torch.empty(0, 24, dtype=BF16, device="cuda")
    y, z = swq.dense_linear(x, w, act=swq.SWQ_ACT_SILU, keep="mx8")
    assert y.shape == (0, 24) and z[0].shape == (0, 24) and z[1].shape == (0, 1)
    dw, dbias = torch.full_like(w, 3.0), torch.full((24,), 3.0, dtype=BF16, device="cuda")
    dx, dw, dbias = swq.dense_linear_backward(dout, x, w, z, act=swq.SWQ_ACT_SILU, dw=dw, dbias=dbias)
    assert dx.shape == (0, 40) and not dw.any() and not dbias.any()


def test_infinities_stay_in_their_rows():
    """An infinity or NaN of one row of x, or of a column's weights, reaches only that row or column, however the
    sizes end inside a tile."""
    for M, K, N in ((3, 37, 20), (40, 70, 131), (300, 130, 269)):
        x, w, bias, _ = layer(M, K, N, BF16)
        x[M - 1, K - 1] = float("inf")
        w[N - 2, 0] = float("nan")
        say("infinities", M, K, N)
        y = swq.dense_linear(x, w, bias)
        bad = ~torch.isfinite(y)
        assert bad[M - 1].all() and bad[:, N - 2].all() and not bad[:M - 1, :N - 2].any() and not bad[:M - 1, N - 1].any()
        dx, dw, db = swq.dense_linear_backward(normal(1, M, N), x, w)
        bad = ~torch.isfinite(dw)
        assert bad[:, K - 1].all() and not bad[:, :K - 1].any()
        bad = ~torch.isfinite(dx)
        assert bad[:, 0].all() and not bad[:, 1:].any() and torch.isfinite(db).all()


def test_leading_dimensions_and_given_outputs():
    x, w, bias, _ = layer(6, 48, 40, BF16)
    say("leading dimensions")
    out = torch.empty(2, 3, 40, dtype=F32, device="cuda")
    y = swq.dense_linear(x.view(2, 3, 48), w, bias, act=2, out_mode=swq.SWQ_LINEAR_F32, out=out)
    assert y is out and torch.equal(out.view(6, 40), swq.dense_linear(x, w, bias, act=2, out_mode=swq.SWQ_LINEAR_F32))
    _, (c, s) = swq.dense_linear(x.view(2, 3, 48), w, bias, act=2, keep="mx8")
    assert c.shape == (2, 3, 40) and s.shape == (2, 3, 2)
    dout = normal(4, 2, 3, 40)
    dx, dw, db = swq.dense_linear_backward(dout, x.view(2, 3, 48), w, (c, s), act=2)
    flat = swq.dense_linear_backward(dout.view(6, 40), x, w, (c.view(6, 40), s.view(6, 2)), act=2)
    assert dx.shape == (2, 3, 48) and torch.equal(dx.view(6, 48), flat[0])
    assert torch.equal(dw, flat[1]) and torch.equal(db, flat[2])


def step(x, w, bias, dout):
    y, z = swq.dense_linear(x, w, bias, act=swq.SWQ_ACT_GELU, keep="mx8")
    return (y, *z, *swq.dense_linear_backward(dout, swq.mx8_quantize(x), w, z, act=swq.SWQ_ACT_GELU))


@pytest.mark.parametrize("M,K,N", [(1, 300, 200), (37, 517, 1001), (300, 256, 512), (1000, 1024, 768)])
def test_repeats_streams_and_graphs(M, K, N):
    """The same bits again, on another stream, and from a graph that is replayed on new inputs with eager
    calls of other sizes on its stream in between."""
    x, w, bias, _ = layer(M, K, N, BF16)
    dout = normal(8, M, N)
    say("repeats, streams, graphs", M, K, N)
    want = step(x, w, bias, dout)
    again = step(x, w, bias, dout)
    assert all(torch.equal(a, b) for a, b in zip(want, again))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        other = step(x, w, bias, dout)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, other))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        held = step(x, w, bias, dout)
    torch.cuda.synchronize()
    for i in range(3):
        x.copy_(normal(20 + i, M, K))
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            g.replay()
        torch.cuda.synchronize()
        for a in held:
            assert not torch.equal(a, torch.zeros_like(a)) or a.dtype == torch.uint8
        got = [a.clone() for a in held]
        with torch.cuda.stream(st):
            step(normal(1, 50, K), w, bias, normal(2, 50, N))      # uses the stream's workspace
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(step(x, w, bias, dout), got))
