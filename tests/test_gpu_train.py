"""8-bit checkpoints, the SwiGLU with checkpoints, the router's balance loss and
gradient on the GPU against their plain 64-bit forms (dense_reference), and a
training step of a routed layer made of them."""
import numpy as np
import pytest
import torch

import dense_reference as ref
import quantized_swiglu_forward_amd as swq
from gpu_helpers import say
from test_gpu_dense import BF16, F16, F32, normal

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------- checkpoints ----

@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("R,K", [(1, 1), (1, 32), (3, 31), (5, 33), (7, 2048), (2, 70), (33, 97), (65, 1056), (130, 64)])
def test_checkpoint(R, K, dtype):
    x = torch.randn(R, K, generator=torch.Generator().manual_seed(R + K))
    x = (x * torch.exp2(torch.randint(-12, 12, (R, 1), generator=torch.Generator().manual_seed(K)).float())).to(dtype).cuda()
    say("checkpoint", R, K, dtype)
    codes, scales = swq.mx8_quantize(x)
    qc, qs = ref.mx8(x)
    assert np.array_equal(scales.cpu().numpy(), qs) and np.array_equal(codes.cpu().numpy(), qc)
    want = ref.mx8_values(codes, scales)
    for out in (BF16, F16, F32):
        v = swq.mx8_dequantize(codes, scales, out)
        ref.close(v, want.clamp(-65504.0, 65504.0) if out == F16 else want,
                  ref.rounding(want, out) if out == F16 else 0 * want, f"values {out}")


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_checkpoint_borders(dtype):
    """Ties, the step's border at 127.5, zeros of both signs, the type's smallest and largest values, infinities, NaN."""
    fi = torch.finfo(dtype)
    rows = [[64.0, 0.5, 1.5, 2.5, -0.5, -1.5, 0.25, 0.75] * 4,
            [127.0, 126.5, -3.5, 3.5] * 8, [127.5, 1.0, -2.0, 3.0] * 8, [127.25, 1.0, -2.0, 3.0] * 8,
            [fi.max, -fi.max, fi.tiny, 0.0] * 8, [fi.tiny, fi.tiny / 2, -fi.tiny, 0.0] * 8,
            [fi.smallest_normal * fi.eps, 0.0] * 16, [float("inf")] + [1.0] * 31, [1.0] * 31 + [float("nan")],
            [0.0, -0.0] * 16]
    x = torch.tensor(rows, dtype=torch.float64).to(dtype).cuda()
    say("checkpoint borders", dtype)
    codes, scales = swq.mx8_quantize(x)
    qc, qs = ref.mx8(x)
    assert np.array_equal(scales.cpu().numpy(), qs) and np.array_equal(codes.cpu().numpy(), qc)
    v = swq.mx8_dequantize(codes, scales, F32)
    assert torch.isnan(v[7:9]).all() and not torch.isnan(v[:7]).any() and not v[9].any()


def test_every_scale():
    codes = torch.tensor([[0, 1, -1, 127, -127, -128, 64, 5]], dtype=torch.int8).repeat(256, 1).cuda()
    scales = torch.arange(256).to(torch.uint8)[:, None].cuda()
    say("every scale")
    want = ref.mx8_values(codes, scales)
    for dtype in (F32, BF16, F16):
        v = swq.mx8_dequantize(codes, scales, dtype)
        w = (want.clamp(-65504.0, 65504.0) if dtype == F16 else want).float().to(dtype)   # binary16 saturates
        assert torch.equal(torch.nan_to_num(v.cpu(), nan=-1.0, posinf=-2.0, neginf=-3.0),
                           torch.nan_to_num(w, nan=-1.0, posinf=-2.0, neginf=-3.0)), dtype


def test_checkpoint_past_32_bits():
    """More than 2^32 elements, rows of an odd length: the last rows against the same rows alone."""
    R, K = (1 << 17) + 5, 33001
    say("checkpoint past 32 bits")
    x = torch.zeros(R, K, dtype=BF16, device="cuda")
    tail = normal(5, 3, K)
    x[-3:] = tail
    codes, scales = swq.mx8_quantize(x)
    c, s = swq.mx8_quantize(tail)
    assert torch.equal(codes[-3:], c) and torch.equal(scales[-3:], s) and not codes[:-3].any()
    out = swq.mx8_dequantize(codes, scales, BF16, out=x)
    assert torch.equal(out[-3:], swq.mx8_dequantize(c, s, BF16)) and not out[:-3].any()


# ------------------------------------------------------------------ SwiGLU ----

@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("R,K", [(1, 1), (1, 768), (3, 33), (6, 768), (17, 1001), (130, 264)])
def test_swiglu(R, K, dtype):
    gate, up, dh = (normal(i + R + K, R, K, dtype=dtype, scale=s) for i, s in enumerate((3.0, 2.0, 1.0)))
    say("swiglu", R, K, dtype)
    hidden, g8, u8 = swq.swiglu(gate, up, keep=True)
    assert torch.equal(hidden, swq.swiglu(gate, up))
    for x, (c, s) in ((gate, g8), (up, u8)):
        qc, qs = swq.mx8_quantize(x)
        assert torch.equal(c, qc) and torch.equal(s, qs)
    want = ref.act(ref.wide(gate), 2) * ref.wide(up)
    ref.close(hidden, want, ref.rounding(want, dtype) * 1.01 + 2.0 ** -20 * want.abs(), "hidden")
    for g, u, wg, wu in ((g8, u8, ref.mx8_values(*g8), ref.mx8_values(*u8)), (gate, up, ref.wide(gate), ref.wide(up)),
                         (g8, up, ref.mx8_values(*g8), ref.wide(up))):
        dgate, dup, again = swq.swiglu_backward(dh, g, u, hidden=True)
        pair = swq.swiglu_backward(dh, g, u)
        assert torch.equal(pair[0], dgate) and torch.equal(pair[1], dup)
        d = ref.wide(dh)
        for got, want, off in ((dgate, d * wu * ref.slope(wg, 2), ref.SLOPE_ERR * (d * wu).abs()),
                               (dup, d * ref.act(wg, 2), 2.0 ** -20 * (d * wg).abs()),
                               (again, ref.act(wg, 2) * wu, 2.0 ** -20 * (wg * wu).abs())):
            ref.close(got, want, ref.rounding(want, dtype) * 1.01 + off, "swiglu gradient")


def test_swiglu_gradient_against_differences():
    R, K = 3, 40
    gate, up, dh = (normal(i + 70, R, K, dtype=F16) for i in range(3))
    say("swiglu differences")
    dgate, dup = swq.swiglu_backward(dh, gate, up)
    g, u, d, h = ref.wide(gate), ref.wide(up), ref.wide(dh), 1e-5
    by_gate = d * u * (ref.act(g + h, 2) - ref.act(g - h, 2)) / (2 * h)
    by_up = d * ref.act(g, 2)
    ref.close(dgate, by_gate, ref.rounding(by_gate, F16) * 1.01 + 1e-6 + ref.SLOPE_ERR * (d * u).abs(), "dgate")
    ref.close(dup, by_up, ref.rounding(by_up, F16) * 1.01 + 1e-6, "dup")


def test_swiglu_empty_and_far():
    say("swiglu empty and far")
    e = torch.empty(0, 64, dtype=BF16, device="cuda")
    hidden, g8, u8 = swq.swiglu(e, e, keep=True)
    assert hidden.shape == (0, 64) and g8[1].shape == (0, 2) and swq.swiglu_backward(e, g8, u8)[0].shape == (0, 64)
    far = torch.tensor([[300.0, -300.0, 3e38, -3e38, 0.0, -0.0]], dtype=BF16, device="cuda")
    one = torch.ones_like(far)
    dgate, dup = swq.swiglu_backward(one, far, one)
    assert dgate.float().tolist() == [[1.0, 0.0, 1.0, 0.0, 0.5, 0.5]]
    assert torch.equal(dup, torch.where(far > 0, far, torch.zeros_like(far)))


# ------------------------------------------------------------------ router ----

def choice(T, E, k, dtype, seed=0, hole=False):
    g = torch.Generator().manual_seed(seed + T + E)
    logits = (2.0 * torch.randn(T, E, generator=g)).to(dtype)
    if hole:                                  # masked experts, rows of nothing else, a NaN, an infinity
        logits[torch.rand(T, E, generator=g) < 0.4] = float("-inf")
        logits[::5] = float("-inf")
        logits[1 % T, 0] = float("nan")
        logits[2 % T, E - 1] = float("inf")
    return logits.cuda(), torch.randn(T, k, generator=g).cuda()


ROUTERS = [(1, 1, 1), (1, 8, 2), (3, 64, 6), (33, 7, 7), (65, 64, 4), (130, 100, 8), (300, 256, 8), (1027, 33, 3),
           (40, 417, 10), (9, 1024, 64)]


@pytest.mark.parametrize("scoring", range(4))
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("T,E,k", ROUTERS)
@pytest.mark.parametrize("hole", [False, True])
def test_router(T, E, k, dtype, scoring, hole):
    logits, dw = choice(T, E, k, dtype, hole=hole)
    ids, weights = swq.route(logits, k, scoring)
    say("router", T, E, k, dtype, scoring, hole)
    loss, counts, slopes = swq.balance_loss(logits, ids, scoring)
    wl, wc, ws = ref.balance(logits, ids, scoring)
    assert torch.equal(counts.cpu().long(), wc)
    ref.close(loss, wl, 2.0 ** -20 * wl.abs() + 1e-30, "loss")
    ref.close(slopes, ws, 2.0 ** -23 * ws, "slopes")
    dw = torch.where(ids < 0, torch.full_like(dw, float("nan")), dw)         # not read where no expert is
    dloss = torch.full((), 0.3 * T, device="cuda")
    for a, b, c in ((dw, slopes, dloss), (dw, None, None), (None, slopes, None)):
        got = swq.route_backward(logits, ids, a, scoring, slopes=b, dloss=c)
        want, tol = ref.route_backward(logits, ids, a, b, float(c) if c is not None else 1.0, scoring)
        ref.close(got, want, tol + ref.rounding(want, dtype) * 1.01, "dlogits")


@pytest.mark.parametrize("scoring", range(4))
def test_router_other_ids(scoring):
    """Ids that no router gives: the same expert twice, ids outside the experts, tokens without a slot, an
    expert whose logit is -inf."""
    T, E, k = 40, 12, 5
    logits, dw = choice(T, E, k, F32, seed=3)
    ids = torch.randint(-3, E + 3, (T, k), generator=torch.Generator().manual_seed(1)).to(torch.int32)
    ids[3] = ids[3, 0] = 4
    ids[7] = -1
    ids[8] = E
    logits[9, ids[9].clamp(0, E - 1).long().cuda()] = float("-inf")
    ids = ids.cuda()
    say("router, other ids", scoring)
    loss, counts, slopes = swq.balance_loss(logits, ids, scoring)
    wl, wc, ws = ref.balance(logits, ids, scoring)
    assert torch.equal(counts.cpu().long(), wc)
    ref.close(loss, wl, 2.0 ** -20 * wl.abs(), "loss")
    got = swq.route_backward(logits, ids, dw, scoring, slopes=slopes)
    want, tol = ref.route_backward(logits, ids, dw, slopes, 1.0, scoring)
    ref.close(got, want, tol, "dlogits")
    assert not got[7].any() and not got[8].any()


@pytest.mark.parametrize("scoring", range(4))
@pytest.mark.parametrize("low", [0.0, -150.0, -3000.0])
def test_router_gradient_against_differences(scoring, low):
    """Against central differences of the 64-bit loss and weights; logits far below zero too (sigmoids that underflow)."""
    T, E, k = 3, 6, 2
    logits, dw = choice(T, E, k, F32, seed=11)
    logits = logits + low
    ids, _ = swq.route(logits, k, scoring)
    say("router differences", scoring, low)
    _, _, slopes = swq.balance_loss(logits, ids, scoring)
    got = swq.route_backward(logits, ids, dw, scoring, slopes=slopes)
    v, ix, ok = ref.wide(logits), ids.cpu().long(), torch.ones(T, k, dtype=torch.bool)
    h, d = 1e-5, torch.zeros(T, E).double()
    for t in range(T):
        for e in range(E):
            for sign in (1, -1):
                moved = v.clone()
                moved[t, e] += sign * h
                f = (ref.shares(moved, scoring) * ref.wide(slopes)).sum()
                f = f + (ref.route_weights(moved, ix, ok, scoring) * ref.wide(dw)).sum()
                d[t, e] += sign * float(f) / (2 * h)
    # h^2 / 6 of a third derivative below 4 |terms|, and 2^-52 |value| / h, together below 1e-9 of terms below 20; at
    # low logits the moved argument is rounded too: 2^-53 3000 / h
    want, tol = ref.route_backward(logits, ids, dw, slopes, 1.0, scoring)
    ref.close(got, d, tol + 1e-8 + 1e-12 * abs(low) / h, "dlogits")


def test_balance_no_tokens_and_no_slots():
    say("balance, empty")
    loss, counts, slopes = swq.balance_loss(torch.empty(0, 9, device="cuda"), torch.empty(0, 2, dtype=torch.int32, device="cuda"))
    assert float(loss) == 0.0 and not counts.any() and not slopes.any()
    logits, ids = normal(1, 50, 9, dtype=F32), torch.full((50, 2), -1, dtype=torch.int32, device="cuda")
    loss, counts, slopes = swq.balance_loss(logits, ids)
    assert float(loss) == 0.0 and not counts.any() and not slopes.any()
    assert not swq.route_backward(logits, ids, normal(2, 50, 2, dtype=F32), slopes=slopes).any()


def test_balance_is_one_when_even():
    """All experts alike and equally often chosen: the loss is 1."""
    T, E = 4096, 8
    say("balance, even")
    ids = (torch.arange(T * 2, device="cuda") % E).to(torch.int32).view(T, 2)
    loss, counts, _ = swq.balance_loss(torch.zeros(T, E, device="cuda"), ids)
    assert abs(float(loss) - 1.0) < 2.0 ** -20 and bool((counts == T * 2 // E).all())


@pytest.mark.parametrize("T", [100, 70000])
def test_router_repeats_streams_and_graphs(T):
    E, k = 64, 6
    logits, dw = choice(T, E, k, BF16)

    def run():
        ids, w = swq.route(logits, k)
        loss, counts, slopes = swq.balance_loss(logits, ids)
        return loss, counts, slopes, swq.route_backward(logits, ids, dw, slopes=slopes)

    say("router repeats, streams, graphs", T)
    want = run()
    assert all(torch.equal(a, b) for a, b in zip(want, run()))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        other = run()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, other))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        held = run()
    for i in range(3):
        logits.copy_(normal(30 + i, T, E))
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            g.replay()
        torch.cuda.synchronize()
        got = [a.clone() for a in held]
        assert all(torch.equal(a, b) for a, b in zip(run(), got))


# ---------------------------------------------------------- the whole layer ----

def test_training_step_of_a_routed_layer():
    """Router logits by dense_linear, route, balance_loss, the gradients back to the router's weight and the layer's input,
    and a dense SwiGLU MLP beside it from 8-bit checkpoints, against autograd in 64 bits.  The chain
    rounds to bf16 five times (2^-8 each) and the checkpoints move gate, up and x by up to 1/127 of a
    block's largest value, in norm below 2^-7 each: 8 of those in quadrature stay below 0.03."""
    T, H, I, E, k = 96, 160, 200, 16, 4
    x, dy = normal(1, T, H), normal(2, T, H)
    wr, br = normal(3, E, H, scale=2 * H ** -0.5), normal(4, E, scale=0.1)
    wg, wu, wd = normal(5, I, H, scale=H ** -0.5), normal(6, I, H, scale=H ** -0.5), normal(7, H, I, scale=I ** -0.5)
    dweights = normal(8, T, k, dtype=F32)
    say("training step")
    logits = swq.dense_linear(x, wr, br, out_mode=swq.SWQ_LINEAR_F32)
    ids, weights = swq.route(logits, k, swq.SWQ_ROUTE_SOFTMAX_CHOSEN)
    loss, counts, slopes = swq.balance_loss(logits, ids, swq.SWQ_ROUTE_SOFTMAX_CHOSEN)
    dlogits = swq.route_backward(logits, ids, dweights, swq.SWQ_ROUTE_SOFTMAX_CHOSEN, slopes=slopes)
    x8 = swq.mx8_quantize(x)
    dx_r, dwr, dbr = swq.dense_linear_backward(dlogits.to(BF16), x8, wr)
    gate, up = swq.dense_linear(x, wg), swq.dense_linear(x, wu)
    hidden, g8, u8 = swq.swiglu(gate, up, keep=True)
    y = swq.dense_linear(hidden, wd, residual=x)
    dgate, dup, again = None, None, None
    dh, _, _ = swq.dense_linear_backward(dy, hidden, wd, want=(True, False, False))
    dgate, dup, again = swq.swiglu_backward(dh, g8, u8, hidden=True)
    _, dwd, _ = swq.dense_linear_backward(dy, again, wd, want=(False, True, False))
    dx_g, dwg, _ = swq.dense_linear_backward(dgate, x8, wg)
    dx_u, dwu, _ = swq.dense_linear_backward(dup, x8, wu)
    dx = dx_r.float() + dx_g.float() + dx_u.float() + dy.float()

    leaf = [ref.wide(t).requires_grad_(True) for t in (x, wr, br, wg, wu, wd)]
    X, WR, BR, WG, WU, WD = leaf
    lo = X @ WR.t() + BR
    ix = ids.cpu().long()
    f = torch.bincount(ix.reshape(-1), minlength=E).double() / ix.numel()
    bal = E * (f * torch.softmax(lo, -1).mean(0)).sum()
    w = torch.softmax(lo.gather(1, ix), -1)
    Y = (torch.nn.functional.silu(X @ WG.t()) * (X @ WU.t())) @ WD.t() + X
    (bal + (w * ref.wide(dweights)).sum() + (Y * ref.wide(dy)).sum()).backward()
    assert torch.equal(counts.cpu().long(), torch.bincount(ix.reshape(-1), minlength=E))
    for name, got, want in (("loss", loss, bal), ("weights", weights, w), ("y", y, Y), ("dx", dx, X.grad), ("dwr", dwr, WR.grad),
                            ("dbr", dbr, BR.grad), ("dwg", dwg, WG.grad), ("dwu", dwu, WU.grad), ("dwd", dwd, WD.grad)):
        want = want.detach()
        rel = float((ref.wide(got) - want).norm() / want.norm())
        assert rel < 0.03, (name, rel)
