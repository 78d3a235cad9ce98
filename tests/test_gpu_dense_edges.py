"""Ends of what the products with 16-bit weights and the router's gradient take, on the GPU: values past the type's largest,
masked experts, the most rows, operands that are not read, the balance loss of many tokens, outputs however allocated."""
import pytest
import torch

import dense_reference as ref
import quantized_swiglu_forward_amd as swq
from gpu_helpers import say
from test_gpu_dense import BF16, F16, F32, normal

pytestmark = pytest.mark.gpu

ACTS = [swq.SWQ_ACT_RELU, swq.SWQ_ACT_SILU, swq.SWQ_ACT_GELU, swq.SWQ_ACT_GELU_TANH]


@pytest.mark.parametrize("M,N", [(5, 40), (150, 200)])
@pytest.mark.parametrize("act", ACTS)
def test_pre_activations_past_binary16(act, M, N):
    """z of +-72000 is an infinity in binary16; its derivatives are 1 and 0 all the same (act' is within 2^-60 of them
    from |z| = 50 on), as they are from a checkpoint, which holds such values."""
    K = 16
    x, w = normal(1, M, K, dtype=F16), torch.full((N, K), 45.0, dtype=F16, device="cuda")
    x[0], x[1], x[M - 1] = 100.0, -100.0, 100.0
    dout = normal(2, M, N, dtype=F16)
    say("past binary16", act, M, N)
    out, z = swq.dense_linear(x, w, act=act, keep="same", out_mode=swq.SWQ_LINEAR_F32)
    want = ref.act(ref.wide(x) @ ref.wide(w).t(), act)
    assert torch.isfinite(out).all() and torch.isinf(z[0]).all() and torch.isinf(z[1]).all()
    assert float(out[0].min()) == 72000.0 and float(out[1].abs().max()) == 0.0 == float(want[1].abs().max())
    wz = ref.wide(z).clamp(-72000.0, 72000.0)
    got = dict(zip(("dx", "dw", "dbias"), swq.dense_linear_backward(dout, x, w, z, act=act)))
    for name, (v, tol) in ref.backward(dout, ref.wide(x), w, wz, act, F16).items():
        ref.close(got[name], v, tol, name)
    _, z8 = swq.dense_linear(x, w, act=act, keep="mx8")
    dx8 = swq.dense_linear_backward(dout, x, w, z8, act=act)[0]
    for row in (0, 1, M - 1):
        assert torch.equal(dx8[row], got["dx"][row])


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_slopes_at_infinities(act, dtype):
    """A kept z of +-inf, next to the type's largest values: 1 and 0; a NaN stays one.  dbias of one row is dz itself."""
    top = torch.finfo(dtype).max
    z = torch.tensor([[float("inf"), float("-inf"), top, -top, float("nan"), 0.0, 1.0, -1.0, 60.0, -200.0]], dtype=dtype,
                     device="cuda")
    dout, w = torch.full_like(z, 3.0), torch.zeros(z.shape[1], 8, dtype=dtype, device="cuda")
    say("slopes at infinities", act, dtype)
    db = swq.dense_linear_backward(dout, None, w, z, act=act, want=(False, False, True))[2].tolist()
    assert db[:4] == [3.0, 0.0, 3.0, 0.0] and db[4] != db[4] and db[8:] == [3.0, 0.0], db
    want = 3.0 * ref.slope(torch.tensor([0.0, 1.0, -1.0]).double(), act)
    ref.close(torch.tensor(db[5:8]), want, 3.0 * ref.SLOPE_ERR + ref.rounding(want, dtype) * 1.01)


@pytest.mark.parametrize("scoring", range(4))
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("T,E,k", [(1, 8, 3), (33, 7, 4), (70, 100, 20), (40, 417, 10)])
def test_slots_of_masked_experts(T, E, k, dtype, scoring):
    """A slot whose expert's logit is -inf or NaN has the weight 0 whatever the others are: what stands in its dweights is
    not read as a number."""
    logits = normal(T + E, T, E, dtype=dtype, scale=2.0)
    ids = torch.stack([torch.randperm(E, generator=torch.Generator().manual_seed(t))[:k] for t in range(T)]).int().cuda()
    dw = normal(5, T, k, dtype=F32)
    hidden = torch.zeros(T, k, dtype=torch.bool, device="cuda")
    hidden[:, 0] = True
    hidden[::3, k - 1] = True
    masked = torch.zeros(T, E, dtype=torch.bool, device="cuda").scatter(1, ids.long(), hidden)
    logits[masked] = float("-inf")
    logits[0, ids[0, 0]] = float("nan")
    slopes = normal(6, E, dtype=F32).abs()
    say("masked experts", T, E, k, dtype, scoring)
    for bad in (float("nan"), float("inf"), float("-inf")):
        for s in (None, slopes):
            got = swq.route_backward(logits, ids, torch.where(hidden, torch.full_like(dw, bad), dw), scoring, slopes=s)
            want = swq.route_backward(logits, ids, torch.where(hidden, torch.zeros_like(dw), dw), scoring, slopes=s)
            assert torch.isfinite(got).all() and torch.equal(got, want), (bad, s is None)
            assert not got[masked].any()


def test_most_rows():
    """2^30 rows: tiles of 2^31 threads, forward and backward, at the first, middle and last rows; all other rows are zeros."""
    M, K, N = 1 << 30, 8, 8
    w = normal(1, N, K)
    say("most rows")
    x = torch.zeros(M, K, dtype=BF16, device="cuda")
    pick = torch.tensor([0, 1, 255, 256, M // 2 - 1, M // 2, M - 257, M - 2, M - 1]).cuda()
    rows = normal(2, len(pick), K)
    x[pick] = rows
    y = swq.dense_linear(x, w)
    want, _, err = ref.linear(rows, w, None, None, 0)
    ref.close(y[pick], want, err + ref.rounding(want, BF16) * 1.01, "out")
    assert int(torch.count_nonzero(y)) == N * len(pick)
    dout = normal(3, len(pick), N)
    y[pick] = dout
    dx, dw, db = swq.dense_linear_backward(y, x, w)
    assert int(torch.count_nonzero(dx)) == K * len(pick)
    for name, (v, tol) in ref.backward(dout, ref.wide(rows), w, None, 0, BF16).items():
        ref.close({"dx": dx[pick], "dw": dw, "dbias": db}[name], v, tol, name)


def test_operands_that_are_not_read():
    """x where dw is not wanted and w where dx is not may lie at any address."""
    M, K, N = 20, 40, 24
    x, w, dout = normal(1, M * K + 1)[1:].view(M, K), normal(2, N * K + 1)[1:].view(N, K), normal(3, M, N)
    say("operands that are not read")
    dx, dw, db = swq.dense_linear_backward(dout, x.clone(), w.clone())
    assert torch.equal(swq.dense_linear_backward(dout, x, w.clone(), want=(True, False, False))[0], dx)
    assert torch.equal(swq.dense_linear_backward(dout, x.clone(), w, want=(False, True, False))[1], dw)
    assert torch.equal(swq.dense_linear_backward(dout, x, w, want=(False, False, True))[2], db)
    for want, xs, ws in (((True, False, False), x, w), ((False, True, False), x, w), ((True, True, True), x, w.clone()),
                         ((True, True, True), x.clone(), w)):
        with pytest.raises(swq.SwigluQError):
            swq.dense_linear_backward(dout, xs, ws, want=want)
    zeros = swq.dense_linear_backward(dout[:0], x[:0], w, want=(False, True, True))
    assert zeros[1].shape == (N, K) and not zeros[1].any() and not zeros[2].any()


@pytest.mark.parametrize("T,E,k,scoring", [(129, 8, 2, 0), (70003, 300, 6, 1), ((1 << 24) + 100, 8, 2, 0), (3000001, 4, 1, 3),
                                           (1 << 20, 256, 8, 2)])
def test_balance_loss_of_many_tokens(T, E, k, scoring):
    """The loss where many blocks share the tokens.  A block has max(32, T / 256) of them and adds them in 32 groups (8 from 257
    experts on) one by one; behind that come at most 2 additions between the groups of a wave, 7 between waves and 8 between
    blocks, the rest is in 64 bits.  So a sum of p is off by that many 2^-24 of itself, and p by 2^-20 as in the router's
    other tests.  Each block counts for far more than that: a sum without any one of them lies outside."""
    g = torch.Generator(device="cuda").manual_seed(1)
    logits = torch.randn(T, E, generator=g, device="cuda")
    ids, _ = swq.route(logits, k, scoring)
    say("balance loss of many tokens", T, E, k, scoring)
    loss, counts, slopes = swq.balance_loss(logits, ids, scoring)
    again = swq.balance_loss(logits, ids, scoring)
    assert all(torch.equal(a, b) for a, b in zip((loss, counts, slopes), again))
    wc = torch.bincount(ids.reshape(-1).long(), minlength=E)
    assert torch.equal(counts.long(), wc)
    rows = max(32, -(-T // 256))
    share = torch.zeros(-(-T // rows), dtype=torch.float64, device="cuda")       # of each block
    for t in range(0, T, rows * 16):
        v = logits[t:t + rows * 16].double()
        p = torch.softmax(v, -1) if scoring < 2 else torch.sigmoid(v)
        p = p @ wc.double() / p.sum(-1)
        share[t // rows:t // rows + -(-len(p) // rows)] = torch.nn.functional.pad(p, (0, -len(p) % rows)).view(-1, rows).sum(-1)
    share *= E / (T * k) / T
    want, tol = float(share.sum()), None
    adds = -(-rows // (32 if E <= 256 else 8)) + 2 + 7 + 8
    tol = (adds * 2.0 ** -24 + 2.0 ** -20) * want
    assert abs(float(loss) - want) <= tol
    assert float(share.min()) > 3.0 * tol                    # (a planted mistake: any block left out)
    by = E / (T * k) / T
    ref.close(slopes, wc.cpu().double() * by, 2.0 ** -23 * wc.cpu().double() * by, "slopes")


def test_outputs_however_allocated(monkeypatch):
    """Outputs are the same tensors (shape, strides, type, device, values) whether the short way to torch's allocator made them
    or its public one, on the current stream and another, with and without inference mode."""
    M, K, N, E, k = 40, 70, 33, 9, 3
    x, w, b, dout = normal(1, M, K), normal(2, N, K), normal(3, N), normal(4, M, N)
    gate, up = normal(5, 2, 3, 40), normal(6, 2, 3, 40)
    logits, e = normal(7, M, E), torch.empty(0, K, dtype=BF16, device="cuda")
    say("outputs however allocated")

    def run():
        y, z = swq.dense_linear(x, w, b, act=swq.SWQ_ACT_SILU, keep="mx8")
        y2, z2 = swq.dense_linear(x, w, b, act=swq.SWQ_ACT_SILU, keep="same", out_mode=swq.SWQ_LINEAR_F32)
        h, g8, u8 = swq.swiglu(gate, up, keep=True)
        ids, _ = swq.route(logits, k)
        x8 = swq.mx8_quantize(x)
        out = [y, *z, y2, z2, *x8, swq.mx8_dequantize(*x8), h, *g8, *u8, *swq.swiglu_backward(h, g8, u8, hidden=True),
               *swq.dense_linear_backward(dout, x8, w, z, act=swq.SWQ_ACT_SILU), *swq.balance_loss(logits, ids),
               swq.route_backward(logits, ids, slopes=swq.balance_loss(logits, ids)[2]),
               swq.dense_linear(e, w), *swq.mx8_quantize(e)]
        torch.cuda.synchronize()
        return out

    def public(shape, stride, dtype):
        return torch.empty_strided(shape, stride, dtype=dtype, device="cuda")

    short = run()
    with torch.inference_mode():
        quiet = run()
    monkeypatch.setattr(swq, "_fresh", public)
    want = run()
    with torch.inference_mode():
        assert [t.is_inference() for t in quiet] == [t.is_inference() for t in run()]
    with torch.cuda.stream(torch.cuda.Stream()):
        other = run()
    for got in (short, quiet, other):
        assert len(got) == len(want)
        for a, b_ in zip(got, want):
            assert (a.shape, a.stride(), a.dtype, a.device) == (b_.shape, b_.stride(), b_.dtype, b_.device)
            assert a.is_contiguous() and torch.equal(a, b_)
