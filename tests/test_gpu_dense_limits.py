"""Far offsets, shared workspaces, unusual calls of the products with 16-bit weights, the checkpoints and the
router's loss and gradient on the GPU."""
import pytest
import torch

import dense_reference as ref
import quantized_swiglu_forward_amd as swq
from gpu_helpers import say
from test_gpu_dense import BF16, F16, F32, normal
from test_gpu_train import choice

pytestmark = pytest.mark.gpu


def test_outputs_past_32_bits():
    """More than 2^32 outputs and bytes of x: the last rows against the same rows alone, and a column far out."""
    M, K, N = (1 << 20) + 70, 2056, 4100
    say("outputs past 32 bits")
    x = torch.zeros(M, K, dtype=BF16, device="cuda")
    x[-40:] = normal(1, 40, K)
    w, bias = normal(2, N, K, scale=K ** -0.5), normal(3, N)
    y = swq.dense_linear(x, w, bias, act=swq.SWQ_ACT_SILU)
    assert torch.equal(y[0], y[M - 41])
    want = swq.dense_linear(torch.cat([x[:88], x[-40:]]), w, bias, act=swq.SWQ_ACT_SILU)
    # (the same tiles: one row's sums do not depend on the others)
    assert float((y[-40:].float() - want[-40:].float()).abs().max()) <= 2.0 ** -7 * float(want.abs().max())
    assert float((y[:1].float() - want[:1].float()).abs().max()) <= 2.0 ** -7 * float(want.abs().max())


def test_inner_indexes_past_32_bits():
    """dW over a dout of more than 4 GiB, its last rows alone not zero; dx of the same rows; dbias."""
    M, K, N = 270000, 24, 8200
    say("inner indexes past 32 bits")
    dout = torch.zeros(M, N, dtype=BF16, device="cuda")
    dout[-5:] = normal(1, 5, N)
    x, w = normal(2, M, K), normal(3, N, K)
    dx, dw, db = swq.dense_linear_backward(dout, x, w)
    wx, wdw, wdb = swq.dense_linear_backward(dout[-5:].contiguous(), x[-5:].contiguous(), w)
    for got, want in ((dx[-5:], wx), (dw, wdw), (db, wdb)):
        assert float((got.float() - want.float()).abs().max()) <= 2.0 ** -7 * float(want.abs().max())
    assert not dx[:-5].any()


def test_long_rows():
    """The longest rows: K = 2^20 inputs, and N = 2^20 outputs, with odd neighbours."""
    say("long rows")
    for M, K, N in ((3, 1 << 20, 9), (70, (1 << 20) - 1, 4), (2, 9, 1 << 20), (67, 12, (1 << 20) - 3)):
        x, w = normal(M, M, K), normal(N, N, K, scale=K ** -0.5)
        y = swq.dense_linear(x, w, out_mode=swq.SWQ_LINEAR_F32)
        want, _, err = ref.linear(x, w, None, None, 0)
        ref.close(y, want, err + ref.rounding(want, F32), f"{M} {K} {N}")
        dout = normal(5, M, N)
        got = dict(zip(("dx", "dw", "dbias"), swq.dense_linear_backward(dout, x, w)))
        for name, (v, tol) in ref.backward(dout, ref.wide(x), w, None, 0, BF16).items():
            ref.close(got[name], v, tol, name)


def test_residual_in_place():
    """out may be the residual itself."""
    for M, K, N in ((5, 96, 70), (200, 256, 333), (700, 4096, 256), (1500, 128, 2000)):
        x, w, r = normal(1, M, K), normal(2, N, K, scale=K ** -0.5), normal(3, M, N)
        say("residual in place", M, K, N)
        want = swq.dense_linear(x, w, residual=r, act=swq.SWQ_ACT_SILU)
        got = swq.dense_linear(x, w, residual=r, act=swq.SWQ_ACT_SILU, out=r)
        assert got is r and torch.equal(got, want)


def test_one_dimension_and_empty_leads():
    w, b = normal(1, 12, 40), normal(2, 12)
    x = normal(3, 40)
    say("one dimension")
    y, z = swq.dense_linear(x, w, b, act=swq.SWQ_ACT_GELU, keep="mx8")
    assert y.shape == (12,) and z[0].shape == (12,) and z[1].shape == (1,)
    dx, dw, db = swq.dense_linear_backward(normal(4, 12), x, w, z, act=swq.SWQ_ACT_GELU)
    assert dx.shape == (40,) and dw.shape == (12, 40) and db.shape == (12,)
    c, s = swq.mx8_quantize(x)
    assert c.shape == (40,) and s.shape == (2,) and swq.mx8_dequantize(c, s).shape == (40,)
    h, g8, u8 = swq.swiglu(x, x, keep=True)
    assert h.shape == (40,) and swq.swiglu_backward(x, g8, u8)[0].shape == (40,)
    ids, _ = swq.route(x, 4)
    loss, counts, slopes = swq.balance_loss(x, ids)
    assert loss.shape == () and int(counts.sum()) == 4 and swq.route_backward(x, ids, slopes=slopes).shape == (40,)
    e = torch.empty(2, 0, 40, dtype=BF16, device="cuda")
    assert swq.dense_linear(e, w, b).shape == (2, 0, 12) and swq.mx8_quantize(e)[1].shape == (2, 0, 2)


def test_workspace_that_grows_between_graph_replays():
    """A captured training step keeps its results when eager calls of the same stream make the workspace larger and use
    it between the replays; two graphs share it."""
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    small, other = (90, 133, 200), (300, 96, 65)
    make = {s: (normal(1, s[0], s[1]), normal(2, s[2], s[1], scale=s[1] ** -0.5), normal(3, s[2]), normal(4, s[0], s[2]))
            for s in (small, other, (3000, 1025, 1100))}

    def step(s):
        x, w, b, dout = make[s]
        y, z = swq.dense_linear(x, w, b, act=swq.SWQ_ACT_SILU, keep="mx8")
        return (y, *z, *swq.dense_linear_backward(dout, swq.mx8_quantize(x), w, z, act=swq.SWQ_ACT_SILU))

    say("workspace grows between replays")
    graphs = {}
    with torch.cuda.stream(st):
        for s in (small, other):
            step(s)
    torch.cuda.synchronize()
    for s in (small, other):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            graphs[s] = (g, step(s))
    for i in range(3):
        for s in (small, other):
            make[s][0].copy_(normal(10 + i, s[0], s[1]))
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            for s in (small, other):
                graphs[s][0].replay()
                step((3000, 1025, 1100))
        torch.cuda.synchronize()
        got = {s: [a.clone() for a in graphs[s][1]] for s in (small, other)}
        for s in (small, other):
            assert all(torch.equal(a, b) for a, b in zip(step(s), got[s])), (i, s)


def test_streams_of_their_own():
    """Calls on two streams at once: each has its own workspace."""
    sizes = [(200, 517, 333), (333, 517, 200)]
    data = [(normal(1, M, K), normal(2, N, K, scale=K ** -0.5), normal(3, M, N)) for M, K, N in sizes]

    def step(x, w, dout):
        y, z = swq.dense_linear(x, w, act=swq.SWQ_ACT_GELU, keep="same")
        return (y, z, *swq.dense_linear_backward(dout, x, w, z, act=swq.SWQ_ACT_GELU))

    say("two streams")
    want = [step(*d) for d in data]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in data]
    got = [None, None]
    for _ in range(20):
        for i, (st, d) in enumerate(zip(streams, data)):
            with torch.cuda.stream(st):
                got[i] = step(*d)
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(a, b) for a, b in zip(g, w))


def test_checkpoint_of_the_largest_values():
    """Binary16's largest value comes back within half a step, not as an infinity, also as an operand of dW."""
    say("largest values")
    x = torch.full((2, 64), 65504.0, dtype=F16, device="cuda")
    x[1] = -65504.0
    c, s = swq.mx8_quantize(x)
    v = swq.mx8_dequantize(c, s, F16)
    assert torch.isfinite(v).all() and float((v.float() - x.float()).abs().max()) <= 512
    dout = torch.zeros(2, 8, dtype=F16, device="cuda")
    dout[0] = 2.0 ** -4
    _, dw, _ = swq.dense_linear_backward(dout, (c, s), normal(1, 8, 64, dtype=F16))
    assert torch.isfinite(dw).all() and float((dw.float() - 65504 / 16).abs().max()) <= 32


@pytest.mark.parametrize("T,E,k,scoring", [((1 << 24) + 100, 8, 2, 0), (3000001, 4, 1, 3)])
def test_router_of_many_tokens(T, E, k, scoring):
    """More tokens than one launch of the gradient takes, against the same formulas in 64 bits (sums of T float32 values per
    block: off by at most T / 256 roundings)."""
    say("router of many tokens", T, E, k)
    g = torch.Generator(device="cuda").manual_seed(1)
    logits = torch.randn(T, E, generator=g, device="cuda")
    ids, _ = swq.route(logits, k, scoring)
    loss, counts, slopes = swq.balance_loss(logits, ids, scoring)
    ix = ids.long()
    wc = torch.bincount(ix.reshape(-1), minlength=E)
    assert torch.equal(counts.long(), wc)
    p = torch.softmax(logits.double(), -1) if scoring < 2 else torch.sigmoid(logits.double())
    if scoring >= 2:
        p /= p.sum(-1, keepdim=True)
    want = E * (wc.double() / (T * k) * p.mean(0)).sum()
    assert abs(float(loss) - float(want)) <= T / 256 * 2.0 ** -24 * float(want) + 2.0 ** -20
    d = swq.route_backward(logits, ids, None, scoring, slopes=slopes)
    rows = torch.cat([torch.arange(50), torch.arange(T - 50, T)]).cuda()
    part, tol = ref.route_backward(logits[rows], ids[rows], None, slopes, 1.0, scoring)
    ref.close(d[rows], part, tol + ref.rounding(part, F32), "dlogits")


def test_counts_of_one_expert():
    """Every token with the same expert, and ids that differ by token count only."""
    T, E = 5000, 300
    say("one expert")
    logits, _ = choice(T, E, 3, BF16)
    ids = torch.full((T, 3), 7, dtype=torch.int32, device="cuda")
    loss, counts, slopes = swq.balance_loss(logits, ids)
    wl, wc, ws = ref.balance(logits, ids, 0)
    assert torch.equal(counts.cpu().long(), wc) and int(counts[7]) == 3 * T
    ref.close(loss, wl, 2.0 ** -18 * wl.abs(), "loss")
    dw = torch.ones(T, 3, device="cuda")
    for scoring in range(4):
        got = swq.route_backward(logits, ids, dw, scoring, slopes=slopes)
        want, tol = ref.route_backward(logits, ids, dw, slopes, 1.0, scoring)
        ref.close(got, want, tol + ref.rounding(want, BF16) * 1.01, f"dlogits {scoring}")
