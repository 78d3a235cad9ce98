"""Plain 64-bit forms of the MXFP4 operators, the router and the experts'
MLP, with the error that each result may carry.

Bounds, per element: a float32 sum of n products a_i b_i (exact products) is off
by at most n 2^-23 sum |a_i b_i| (each addition by one unit in the last place
of a partial sum at most), a rounding to a type by half its eps relative to
the value, and what a later product multiplies is carried through it."""
import numpy as np
import torch

MAG = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
# what is lost below a type's normal range: half its smallest subnormal
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}


def unpack(codes):
    c = codes.cpu().numpy().view(np.uint32)
    return ((c[..., None] >> (4 * np.arange(8, dtype=np.uint32))) & 15).reshape(*c.shape[:-1], -1)


def values(codes, scales):
    """float64 values [..., K]."""
    q = unpack(codes)
    v = np.where(q >= 8, -1.0, 1.0) * MAG[q & 7]
    s = scales.cpu().numpy().astype(np.int64)
    f = np.where(s == 255, np.nan, np.ldexp(1.0, s - 127))
    return v * np.repeat(f, 32, -1)


def quantize(x):
    """(codes [rows, K] as numbers 0..15, scale bytes [rows, K/32]) of a tensor, in float64."""
    b = x.detach().cpu().double().numpy().reshape(-1, 32)
    codes, scales = np.zeros(b.shape, np.int64), np.zeros(b.shape[0], np.int64)
    for i, row in enumerate(b):
        top = np.abs(row).max()
        if not np.isfinite(top):
            scales[i] = 255
            continue
        e = -127 if top == 0 else min(127, max(-127, int(np.frexp(top)[1]) - 3))
        a = np.abs(np.ldexp(row, -e))
        d = np.abs(a[:, None] - MAG[None, :])
        near = d == d.min(1, keepdims=True)
        even = near & (np.arange(8) % 2 == 0)
        codes[i] = np.where(even.any(1), even.argmax(1), near.argmax(1)) + 8 * np.signbit(row)
        scales[i] = e + 127
    return codes.reshape(*x.shape), scales.reshape(*x.shape[:-1], -1)


def to64(t):
    return t.detach().cpu().double().numpy()


def dot(x, w, xe=None):
    """(x w^T, its bound): x [m, K] with the error xe, w [n, K]."""
    y = x @ w.T
    size = np.abs(x) @ np.abs(w).T
    err = x.shape[-1] * 2.0 ** -23 * size
    if xe is not None:
        err = err * (1 + 2.0 ** -8) + xe @ np.abs(w).T
    return y, err


def rounded(y, err, dtype):
    return err + HALF_STEP[dtype] * (np.abs(y) + err) + TINY[dtype]


def close(got, y, err, what=""):
    g = to64(got)
    assert g.shape == y.shape, (what, g.shape, y.shape)
    bad = ~(np.abs(g - y) <= err)
    bad &= ~(np.isnan(g) & np.isnan(y)) & ~((g == y) & np.isinf(y))
    if bad.any():
        i = tuple(int(v[0]) for v in np.nonzero(bad))
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} outside, first at {i}: {g[i]} for {y[i]} "
                             f"within {err[i]}")


def mlp(x, wg, wu, wd, hidden_half):
    """(y, bound) of one expert's MLP in float64; hidden_half: half a step of the hidden tensor's rounding."""
    g, ge = dot(x, wg)
    u, ue = dot(x, wu)
    with np.errstate(over="ignore"):
        sg = 1 / (1 + np.exp(-g))
    h = g * sg * u
    # |silu'| <= 1.1; the sigmoid and the two products: 8 units of 2^-23
    he = 1.1 * ge * (np.abs(u) + ue) + (np.abs(g * sg) + 1.1 * ge) * ue + 8 * 2.0 ** -23 * np.abs(h) + 2.0 ** -126
    he = he + hidden_half * (np.abs(h) + he)
    return dot(h, wd, he)


def experts(x, ids, weights, wg, wu, wd, residual, hidden_half):
    """(out, bound): ids and weights as numpy, everything float64."""
    T, k = ids.shape
    E = wg.shape[0]
    y = np.zeros((T, wd.shape[1])) if residual is None else residual.copy()
    size, err = np.abs(y), np.zeros_like(y)
    for t in range(T):
        for j in range(k):
            e = ids[t, j]
            if not 0 <= e < E:
                continue
            p, pe = mlp(x[t:t + 1], wg[e], wu[e], wd[e], hidden_half)
            y[t] += weights[t, j] * p[0]
            err[t] += abs(weights[t, j]) * pe[0]
            size[t] += abs(weights[t, j]) * (np.abs(p[0]) + pe[0])
    return y, err + (k + 1) * 2.0 ** -23 * size


def route(logits, k, scoring):
    """(ids, weights) in float64."""
    v = to64(logits)
    v = np.where(np.isnan(v), -np.inf, np.minimum(v, 3.402823466385288598e38))
    T, E = v.shape
    ids, w = np.full((T, k), -1, np.int64), np.zeros((T, k))
    for t in range(T):
        order = [e for e in np.argsort(-v[t], kind="stable") if v[t, e] > -np.inf]
        chosen = order[:k]
        if not chosen:
            continue
        a = v[t, chosen]
        if scoring < 2:
            over = v[t, order] if scoring == 0 else a
            p = np.exp(a - a[0]) / np.exp(over - a[0]).sum()
        else:
            # sigmoid(a) = e^min(a, 0) / (1 + e^-|a|); the ratio is taken before it underflows
            p = np.exp(np.minimum(a, 0) - (min(a[0], 0) if scoring == 3 else 0)) / (1 + np.exp(-np.abs(a)))
            if scoring == 3:
                p = p / p.sum()
        ids[t, :len(chosen)], w[t, :len(chosen)] = chosen, p
    return ids, w
