"""Mistakes planted in the plain 64-bit forms of the MXFP4 operators, the router
and the experts' MLP: each must leave the bounds that the GPU tests use, and a
float32 computation without a mistake must stay inside them."""
import numpy as np
import pytest
import torch

import mx4_reference as ref

M, K, N, E = 5, 96, 24, 3


def matrix(seed, *shape):
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(-2 ** 31, 2 ** 31, (*shape[:-1], shape[-1] // 8), generator=g).to(torch.int32)
    return codes, torch.randint(119, 126, (*shape[:-1], shape[-1] // 32), generator=g).to(torch.uint8)


def rows(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).bfloat16()


def outside(got, y, err):
    with pytest.raises(AssertionError, match="outside"):
        ref.close(torch.from_numpy(np.asarray(got)), y, err)


# ------------------------------------------------------------ the format ----

FORMAT = {
    "nibbles of a byte swapped": lambda q, s: (q.reshape(*q.shape[:-1], -1, 2)[..., ::-1].reshape(q.shape), s),
    "sign ignored": lambda q, s: (q & 7, s),
    "scale of the next block": lambda q, s: (q, np.roll(s, 1, -1)),
    "exponent off by one": lambda q, s: (q, s + 1),
    "blocks of 16": lambda q, s: (q, np.repeat(s, 2, -1)[..., :s.shape[-1]]),
    "code 7 as 5": lambda q, s: (np.where(q % 8 == 7, q - 1, q), s),
}


@pytest.mark.parametrize("mistake", FORMAT, ids=list(FORMAT))
def test_format(mistake):
    x, (w, s) = ref.to64(rows(1, M, K)), matrix(2, N, K)
    y, err = ref.dot(x, ref.values(w, s))
    good = (x.astype(np.float32) @ ref.values(w, s).astype(np.float32).T).astype(np.float64)
    ref.close(torch.from_numpy(good), y, ref.rounded(y, err, torch.float32))
    q, t = FORMAT[mistake](ref.unpack(w), s.numpy().astype(np.int64))
    v = np.where(q >= 8, -1.0, 1.0) * ref.MAG[q & 7] * np.repeat(np.ldexp(1.0, t - 127), 32, -1)
    outside(x @ v.T, y, ref.rounded(y, err, torch.bfloat16))


# ------------------------------------------------------------ the products ----

PRODUCTS = {
    "last block of K left out": lambda x, w: x[:, :-32] @ w[:, :-32].T,
    "one input twice": lambda x, w: x @ w.T + np.outer(x[:, 40], w[:, 40]),
    "columns one off": lambda x, w: np.roll(x @ w.T, 1, 1),
    "rows one off": lambda x, w: np.roll(x @ w.T, 1, 0),
    "x rounded to four bits": lambda x, w: ref.to64(torch.from_numpy(x).to(torch.float8_e4m3fn).double()) @ w.T,
}


@pytest.mark.parametrize("mistake", PRODUCTS, ids=list(PRODUCTS))
def test_product(mistake):
    x, w = ref.to64(rows(3, M, K)), ref.values(*matrix(4, N, K))
    y, err = ref.dot(x, w)
    outside(PRODUCTS[mistake](x, w), y, ref.rounded(y, err, torch.bfloat16))


# ---------------------------------------------------------- the quantiser ----

def nearest(a):
    """Magnitude codes of the values nearest to a, the lower one on a tie (8: past the format)."""
    return np.abs(a[..., None] - np.append(ref.MAG, 8.0)).argmin(-1)


QUANT = {
    "ties up": lambda a: nearest(a + 2.0 ** -20),
    "ties down": nearest,
    "exponent one too large": lambda a: nearest(a / 2),
    "no saturation": lambda a: nearest(np.where(a > 7, 8.0, a)),
}


@pytest.mark.parametrize("mistake", QUANT, ids=list(QUANT))
def test_quantiser(mistake):
    """Codes are compared exactly: each mistake changes some on ties, borders and large elements."""
    x = torch.tensor([[0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.5, 6.5, 7.5] + [-1.0] * 22], dtype=torch.float64)
    codes, scales = ref.quantize(x)
    assert scales.tolist() == [[127]]
    assert codes[0, :10].tolist() == [0, 2, 2, 4, 4, 6, 6, 7, 7, 7]
    assert (QUANT[mistake](np.abs(x.numpy())[:, :10]) != codes[:, :10]).any()


# -------------------------------------------------------------- the router ----

def softmax(v):
    p = np.exp(v - v.max())
    return p / p.sum()


def test_router():
    lo = torch.tensor([[0.5, 2.0, 2.0, -1.0, float("-inf"), float("nan")]])
    v = lo.numpy().astype(np.float64)[0, :4]
    ids, w = ref.route(lo, 5, 0)
    assert ids.tolist() == [[1, 2, 0, 3, -1]] and w[0, 4] == 0
    assert np.allclose(w[0, :4], softmax(v)[ids[0, :4]], rtol=1e-15)
    ids, w = ref.route(lo, 2, 1)
    assert ids.tolist() == [[1, 2]] and w.tolist() == [[0.5, 0.5]]
    tol = 64 * 2.0 ** -24
    all_, chosen = ref.route(lo, 2, 0)[1], ref.route(lo, 2, 1)[1]
    sig, part = ref.route(lo, 3, 2)[1], ref.route(lo, 3, 3)[1]
    assert np.all(np.abs(all_ - chosen) > tol * chosen)               # softmax over the wrong set
    assert np.all(np.abs(sig - part) > tol * part)                    # the sigmoids' sum forgotten
    assert np.allclose(sig, 1 / (1 + np.exp(-np.array([[2.0, 2.0, 0.5]]))), rtol=1e-15)
    assert np.allclose(part.sum(), 1, rtol=1e-15)


# ------------------------------------------------------------- the experts ----

def layer(x, ids, weights, wg, wu, wd, residual, silu=lambda g: g / (1 + np.exp(-g)), swap=False):
    y = residual.copy()
    for t in range(ids.shape[0]):
        for j in range(ids.shape[1]):
            e = ids[t, j]
            if 0 <= e < wg.shape[0]:
                g, u = x[t] @ wg[e].T, x[t] @ wu[e].T
                y[t] += weights[t, j] * (wd[e] @ (silu(u) * g if swap else silu(g) * u))
    return y


EXPERTS = {
    "gate and up swapped": lambda a: layer(*a, swap=True),
    "gelu's slope in silu": lambda a: layer(*a, silu=lambda g: g / (1 + np.exp(-1.702 * g))),
    "weights one slot off": lambda a: layer(a[0], a[1], np.roll(a[2], 1, 1), *a[3:]),
    "ids one token off": lambda a: layer(a[0], np.roll(a[1], 1, 0), *a[2:]),
    "residual left out": lambda a: layer(*a[:-1], np.zeros_like(a[-1])),
    "a skipped slot as expert 0": lambda a: layer(a[0], np.where(a[1] < 0, 0, a[1]), *a[2:]),
}


@pytest.mark.parametrize("mistake", EXPERTS, ids=list(EXPERTS))
def test_experts(mistake):
    x, res = ref.to64(rows(5, M, K)), ref.to64(rows(6, M, 40))
    ids = np.array([[0, 1], [2, 0], [1, -1], [0, 2], [2, 1]])
    weights = np.random.default_rng(0).uniform(0.2, 1, (M, 2))
    w = [ref.values(*matrix(7 + i, *s)) for i, s in enumerate(((E, 64, K), (E, 64, K), (E, 40, 64)))]
    y, err = ref.experts(x, ids, weights, *w, res, 2.0 ** -8)
    bound = ref.rounded(y, err, torch.bfloat16)
    a = (x, ids, weights, *w, res)
    ref.close(torch.from_numpy(layer(*a)), y, bound)
    outside(EXPERTS[mistake](a), y, bound)
