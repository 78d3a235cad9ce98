"""Plain 64-bit forms of the products with 16-bit weights, the activations, the
8-bit checkpoints, the SwiGLU and the router's loss and gradient, and how far a
result may be off.

The bounds.  u is half a step of the output type relative to the value (bf16 2^-8, binary16 2^-11, float32 2^-24), and
binary16 results below 2^-14 are off by at most half of 2^-24.  A float32 sum of n exact
products in any order is off by at most n 2^-24 sum|terms|; a matrix instruction may round each addition toward zero, so
2^-23 is taken, and two steps for bias and residual.  The activations (hardware exp2 and
reciprocal, 1 ulp each, of an argument that is itself rounded): a sigmoid is off by at most 2^-22 (1 + |t|) of itself,
|t| sigma(t)(1 - sigma(t)) < 0.23; erfc's formula by 1.5e-7 absolute, so a normal
probability by 0.75e-7 < 2^-23.  An activation's value is within 2^-20 |z| (with z sigma(z)'s
factor), its derivative within 2^-19 (1 + ...): the largest factor is |z| sigma' (1 + 0.134 z^2) 1.6 < 2 of the tanh form, times
2^-22 (1 + |t|), t below 20 where sigma' is above 2^-29."""
import math

import numpy as np
import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
SUM = 2.0 ** -23
ACT_ERR, SLOPE_ERR = 2.0 ** -20, 2.0 ** -16


def wide(t):
    return t.detach().cpu().double()


def rounding(y, dtype):
    """How far rounding y to dtype moves it."""
    out = U[dtype] * y.abs()
    return out + 2.0 ** -25 if dtype == torch.float16 else out


def close(got, want, tol, what=""):
    """Elementwise, with NaN and infinities where the reference has them."""
    got, want = wide(got).reshape(want.shape), want
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN in other places"
    assert torch.equal(got[~fine & ~torch.isnan(want)], want[~fine & ~torch.isnan(want)]), f"{what}: other infinities"
    off = (got - want).abs()[fine] - tol.expand_as(want)[fine]
    if off.numel():
        i = int(off.argmax())
        assert off[i] <= 0, (f"{what}: {got[fine][i]:.9g} for {want[fine][i]:.9g}, off by "
                             f"{(got - want).abs()[fine][i]:.3g}, allowed {tol.expand_as(want)[fine][i]:.3g}")


# ------------------------------------------------------------- activations ----

def act(z, a):
    """a: 0 none, 1 relu, 2 silu, 3 gelu, 4 gelu by tanh."""
    if a == 1:
        return z.clamp(min=0.0)
    if a == 2:
        return z * torch.sigmoid(z)
    if a == 3:
        return 0.5 * z * torch.special.erfc(-z * math.sqrt(0.5))
    if a == 4:
        return z * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))
    return z


def slope(z, a):
    if a == 1:
        return (z > 0).double()
    if a == 2:
        s = torch.sigmoid(z)
        return s * (1.0 + z * torch.sigmoid(-z))
    if a == 3:
        return 0.5 * torch.special.erfc(-z * math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if a == 4:
        c = 2.0 * math.sqrt(2.0 / math.pi)
        u = c * (z + 0.044715 * z ** 3)
        return torch.sigmoid(u) + z * torch.sigmoid(u) * torch.sigmoid(-u) * c * (1.0 + 3.0 * 0.044715 * z * z)
    return torch.ones_like(z)


# ------------------------------------------------------------- checkpoints ----

def mx8(x):
    """(codes [R, K], scale bytes [R, ceil(K / 32)]) of a host tensor [R, K], as numpy arrays."""
    v = wide(x).numpy()
    R, K = v.shape
    nb = (K + 31) // 32
    codes, scales = np.zeros((R, K), np.int64), np.zeros((R, nb), np.int64)
    for b in range(nb):
        blk = v[:, 32 * b:32 * b + 32]
        for r in range(R):
            top = np.abs(blk[r]).max()
            if not np.isfinite(top):
                scales[r, b] = 255
                continue
            e = -126 if top == 0 else max(math.frexp(top)[1] - 7, -126)
            if np.rint(math.ldexp(top, -e)) > 127 and e < 121:
                e += 1
            codes[r, 32 * b:32 * b + 32] = np.clip(np.rint(np.ldexp(blk[r], -e)), -127, 127)
            scales[r, b] = e + 133
    return codes, scales


def mx8_values(codes, scales):
    """The 64-bit values of a checkpoint (device or host tensors)."""
    q, b = wide(codes), wide(scales)
    K = q.shape[-1]
    step = torch.where(b == 255, torch.full_like(b, float("nan")), torch.from_numpy(np.ldexp(1.0, b.numpy().astype(int) - 133)))
    return q * step.repeat_interleave(32, -1)[..., :K]


def mx8_half_steps(scales, K):
    b = wide(scales).numpy().astype(int)
    return torch.from_numpy(np.ldexp(0.5, b - 133)).repeat_interleave(32, -1)[..., :K]


# ---------------------------------------------------------------- products ----

def linear(x, w, bias, residual, a):
    """(out, z, how far z's float32 sum may be off) in 64 bits."""
    x, w = wide(x), wide(w)
    z = x @ w.t()
    mass = x.abs() @ w.abs().t()
    if bias is not None:
        z, mass = z + wide(bias), mass + wide(bias).abs()
    err = (x.shape[-1] + 2) * SUM * mass
    out = act(z, a)
    return (out if residual is None else out + wide(residual)), z, err


def linear_tol(z, err, residual, a, out, dtype):
    more = 0.0 if residual is None else U[torch.float32] * (out.abs() + wide(residual).abs())
    return 1.2 * err + (ACT_ERR * z.abs() if a > 1 else 0.0) + more + rounding(out, dtype) * 1.01


def backward(dout, x, w, z, a, dtype):
    """{name: (64-bit gradient, tolerance)} for 64-bit x and z as the call gets them."""
    d, w = wide(dout), wide(w)
    s = slope(z, a) if a else torch.ones_like(d)
    dz = d * s
    off = d.abs() * (SLOPE_ERR if a > 1 else 0.0)                       # of dz in float32
    off16 = off + (rounding(dz, dtype) * 1.01 if a else 0.0)             # of dz as an operand
    M, N = dz.shape
    out = {}
    dx = dz @ w
    out["dx"] = dx, off16 @ w.abs() + (N + 2) * SUM * (dz.abs() @ w.abs()) + rounding(dx, dtype) * 1.01
    dw = dz.t() @ x
    out["dw"] = dw, off16.t() @ x.abs() + (M + 2) * SUM * (dz.abs().t() @ x.abs()) + rounding(dw, dtype) * 1.01
    db = dz.sum(0)
    out["dbias"] = db, off.sum(0) + (M + 2) * 2.0 ** -24 * dz.abs().sum(0) + rounding(db, dtype) * 1.01
    return out


# ------------------------------------------------------------------ router ----

def router_logits(logits):
    """As the router takes them: NaN is -inf, +inf the largest float32."""
    v = wide(logits)
    v = torch.where(torch.isnan(v), torch.full_like(v, float("-inf")), v)
    return v.clamp(max=torch.finfo(torch.float32).max)


def shares(v, scoring):
    """p over each row's experts; 0 for -inf, also in rows of nothing else."""
    if scoring < 2:
        top = v.amax(-1, keepdim=True)
        e = torch.exp(v - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    else:
        top = v.amax(-1, keepdim=True).clamp(max=0.0)
        top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
        e = torch.exp(v.clamp(max=0.0) - top) / (1.0 + torch.exp(-v.abs()))
    s = e.sum(-1, keepdim=True)
    return torch.where(s > 0, e / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(e))


def balance(logits, ids, scoring):
    """(loss, counts, slopes) in 64 bits."""
    v, ids = router_logits(logits), ids.cpu().long()
    T, E = v.shape
    ok = (ids >= 0) & (ids < E)
    live = ok.any(-1)
    counts = torch.bincount(ids[ok], minlength=E)
    N, tokens = int(counts.sum()), int(live.sum())
    if N == 0:
        return torch.zeros(()).double(), counts, torch.zeros(E).double()
    P = shares(v, scoring)[live].sum(0) / tokens
    f = counts.double() / N
    return E * (f * P).sum(), counts, E * f / tokens


def route_weights(v, ids, ok, scoring):
    """The routing weights of given slots as a function of 64-bit logits (0 for slots that do not count)."""
    at = ids.clamp(0, v.shape[-1] - 1)
    lv = torch.where(ok, v.gather(-1, at), torch.full_like(v.gather(-1, at), float("-inf")))
    if scoring == 0:
        return torch.where(ok, shares(v, 0).gather(-1, at), torch.zeros_like(lv))
    if scoring == 2:
        return torch.where(ok, torch.sigmoid(lv), torch.zeros_like(lv))
    return shares(lv, scoring)


def route_backward(logits, ids, dweights, slopes, dloss, scoring):
    """The gradient in 64 bits, by the formulas."""
    v, ids = router_logits(logits), ids.cpu().long()
    T, E = v.shape
    ok = (ids >= 0) & (ids < E)
    live = ok.any(-1, keepdim=True)
    p = shares(v, scoring)
    far = torch.where(torch.isinf(v), torch.zeros_like(v), torch.sigmoid(-v))
    g = torch.zeros_like(v)
    if slopes is not None:
        g = g + torch.where(live, wide(slopes)[None, :] * dloss, torch.zeros_like(v))
    at = ids.clamp(0, E - 1)
    slot = torch.zeros(ids.shape).double()
    if dweights is not None:
        dw = torch.where(ok, wide(dweights), torch.zeros(ids.shape).double())
        if scoring == 0:
            g = g.scatter_add(1, at, dw)
        else:
            w = route_weights(v, ids, ok, scoring)
            slot = w * (dw - (w * dw).sum(-1, keepdim=True)) if scoring in (1, 3) else w * dw
            if scoring >= 2:
                slot = slot * far.gather(1, at)
    d = p * (g - (g * p).sum(-1, keepdim=True))
    if scoring >= 2:
        d = d * far
    d = d.scatter_add(1, at, torch.where(ok & ~torch.isinf(v.gather(1, at)), slot, torch.zeros_like(slot)))
    # every term rounds a few times: 2^-19 of the terms' size is over thirty steps of float32
    mass = p * (g.abs() + (g.abs() * p).sum(-1, keepdim=True))
    mass = mass.scatter_add(1, at, slot.abs() + (0 if dweights is None else route_weights(v, ids, ok, scoring)
                                                 * dw.abs().sum(-1, keepdim=True)))
    return d, 2.0 ** -19 * mass + 1e-37
