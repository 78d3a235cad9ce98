"""Kernels and branches of the MXFP4 operators that the sizes of test_gpu_mx4 do
not reach, against the same 64-bit forms and bounds: K splits of aligned rows,
one row of long K, plans made from offsets (more than 64 experts), scale bytes
over their whole range, a workspace that grows after a capture, and the LDS
poison build on the plan and the K split."""
import numpy as np
import pytest
import torch

import mx4_reference as ref
import quantized_swiglu_forward_amd as swq
from gpu_helpers import say
from test_gpu_mx4 import BF16, F16, F32, HIDDEN, MODE, acts, gen, matrix, moe_case
from test_gpu_mx4_poison import both, poison  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _device():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    swq.lib()
    yield
    torch.cuda.synchronize()


def with_residual(y, err, res):
    """(y + residual, its bound): one more addition in float32."""
    if res is None:
        return y, err
    r = ref.to64(res)
    return y + r, err + 2.0 ** -23 * (np.abs(y) + np.abs(r))


# K splits (tiles on at most half the CUs, K >= 1024): rows of outputs of 8, of 4 and odd
SPLIT = [(64, 2080, 1024), (64, 2080, 1028), (40, 4096, 2049), (200, 1152, 1536), (256, 5632, 256)]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("M,K,N", SPLIT)
def test_linear_k_split(M, K, N, dtype):
    x, (w, s), res = acts(M, M, K, dtype=dtype), matrix(N, N, K), acts(3, M, N, dtype=dtype)
    y, err = ref.dot(ref.to64(x), ref.values(w, s))
    for out, r in ((dtype, None), (F32, None), (dtype, res), (F32, res)):
        say("k split", M, K, N, dtype, out, "residual", r is not None)
        got = swq.mx4_linear(x, w, s, residual=r, out_mode=MODE[out])
        yy, ee = with_residual(y, err, r)
        ref.close(got, yy, ref.rounded(yy, ee, out), f"k split {out}")


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("K,N", [(4160, 130), (2080, 33), (14336, 260)])
def test_one_row_of_long_k(K, N, dtype):
    x, (w, s), res = acts(K, 1, K, dtype=dtype), matrix(N, N, K), acts(3, 1, N, dtype=dtype)
    y, err = ref.dot(ref.to64(x), ref.values(w, s))
    for out, r in ((dtype, None), (F32, res)):
        say("one row", K, N, dtype, out)
        got = swq.mx4_linear(x, w, s, residual=r, out_mode=MODE[out])
        yy, ee = with_residual(y, err, r)
        ref.close(got, yy, ref.rounded(yy, ee, out), f"one row {out}")


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("T,k,E,H,I,Ho", [(1, 4, 8, 2080, 1056, 130), (6, 2, 4, 4096, 96, 64), (3, 3, 5, 96, 2112, 33)])
def test_moe_few_tokens_of_long_k(T, k, E, H, I, Ho, dtype):
    x, ids, weights, ws = moe_case(T, T, k, E, H, I, Ho, dtype)
    res = acts(7, T, Ho, dtype=dtype)
    say("moe of long k", T, k, E, H, I, Ho, dtype)
    got = swq.moe_mlp(x, ids, weights, *ws[0], *ws[1], *ws[2], residual=res, out_mode=swq.SWQ_LINEAR_F32)
    y, err = ref.experts(ref.to64(x), ids.cpu().numpy(), ref.to64(weights), *(ref.values(*t) for t in ws),
                         ref.to64(res), HIDDEN[dtype])
    ref.close(got, y, ref.rounded(y, err, F32), "moe of long k")


# Tokens on both sides of the border between slot by slot (few tokens that share few experts) and by expert,
# the few-row kernels of the latter with one, two and four row tiles.
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("T,k,E,H,I,Ho", [(8, 8, 64, 256, 96, 130), (16, 8, 16, 96, 64, 33), (17, 8, 40, 160, 96, 64),
                                          (33, 4, 12, 96, 352, 70), (2, 64, 64, 64, 32, 40), (3, 64, 70, 64, 32, 40),
                                          (129, 1, 9, 288, 64, 96), (128, 1, 9, 288, 64, 96), (24, 6, 100, 64, 64, 130)])
def test_moe_few_tokens(T, k, E, H, I, Ho, dtype):
    x, ids, weights, ws = moe_case(T + E, T, k, E, H, I, Ho, dtype)
    res = acts(7, T, Ho, dtype=dtype)
    say("moe of few tokens", T, k, E, H, I, Ho, dtype)
    got = swq.moe_mlp(x, ids, weights, *ws[0], *ws[1], *ws[2], residual=res)
    y, err = ref.experts(ref.to64(x), ids.cpu().numpy(), ref.to64(weights), *(ref.values(*t) for t in ws),
                         ref.to64(res), HIDDEN[dtype])
    ref.close(got, y, ref.rounded(y, err, dtype), "moe of few tokens")


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("T,k,E", [(4, 4, 4), (5, 4, 4), (3, 8, 8)])
def test_moe_shared_experts(T, k, E, dtype):
    """Every token to every expert, weights large enough to be read once (sizes on both sides of the border)."""
    H, I, Ho = 2048, 1024, 2048
    x, ids, weights, ws = moe_case(T + E, T, k, E, H, I, Ho, dtype, spread=False)
    say("moe of shared experts", T, k, E, dtype)
    got = swq.moe_mlp(x, ids, weights, *ws[0], *ws[1], *ws[2], out_mode=swq.SWQ_LINEAR_F32)
    y, err = ref.experts(ref.to64(x), ids.cpu().numpy(), ref.to64(weights), *(ref.values(*t) for t in ws), None,
                         HIDDEN[dtype])
    ref.close(got, y, ref.rounded(y, err, F32), "moe of shared experts")


# ------------------------------------------- plans from offsets: 66 experts ----

def taken(offsets, P):
    """The groups that the offsets stand for: the nearest non-decreasing ones within the rows."""
    return np.maximum.accumulate(np.clip(np.array(offsets, np.int64), 0, P))


def offsets_of(kind, P, E):
    g = gen(P + E)
    edges = torch.randint(0, P + 1, (E + 1,), generator=g).sort().values
    if kind == "covering":
        edges[0], edges[-1] = 0, P
    elif kind == "gaps":                       # rows before the first and after the last group
        edges = edges * 3 // 5 + P // 5
    elif kind == "unordered":                  # every third one falls back
        edges[2::3] = edges[2::3] - P // 3
    elif kind == "outside":                    # from below 0 to past the rows
        edges = edges * 2 - P // 2
        edges[0], edges[-1] = -(1 << 31), (1 << 31) - 1
    elif kind == "none":                       # no row has an expert
        edges[:] = P // 2
    elif kind == "one":                        # every row has the last
        edges[:-1], edges[-1] = 0, P
    return edges.to(torch.int32)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("kind", ["covering", "gaps", "unordered", "outside", "none", "one"])
@pytest.mark.parametrize("P,E", [(50, 66), (1000, 66), (4000, 66), (300, 2), (2300, 130)])
def test_grouped_offsets(P, E, kind, dtype):
    """Few rows and tiles, from a plan and from the products' own scan, for every shape that offsets can have."""
    K, N = 96, 70
    x, (w, s) = acts(P, P, K, dtype=dtype), matrix(E, E, N, K)
    off = offsets_of(kind, P, E)
    out = torch.full((P, N), float("nan"), device="cuda")
    say("grouped offsets", P, E, kind, dtype)
    swq.mx4_grouped_linear(x, off.cuda(), w, s, out_mode=swq.SWQ_LINEAR_F32, out=out)
    at, xv, wv = taken(off.tolist(), P), ref.to64(x), ref.values(w, s)
    y, err = np.zeros((P, N)), np.zeros((P, N))
    for e in range(E):
        a, b = at[e], at[e + 1]
        if b > a:
            y[a:b], err[a:b] = ref.dot(xv[a:b], wv[e])
    ref.close(out, y, ref.rounded(y, err, F32) * (y != 0), f"grouped {kind}")


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_grouped_large_tiles_of_a_plan(dtype):
    """More than 64 experts with enough rows and columns each for the largest tiles."""
    E, K, N, each = 66, 64, 2056, 150
    P = E * each
    x, (w, s) = acts(1, P, K, dtype=dtype), matrix(E, E, N, K)
    off = (torch.arange(E + 1) * each).to(torch.int32)
    off[1:-1] += torch.randint(-60, 60, (E - 1,), generator=gen(2)).to(torch.int32)
    say("grouped large tiles of a plan", dtype)
    got = swq.mx4_grouped_linear(x, off.cuda(), w, s, out_mode=swq.SWQ_LINEAR_F32)
    xv, wv = ref.to64(x), ref.values(w, s)
    for e in range(E):
        a, b = int(off[e]), int(off[e + 1])
        y, err = ref.dot(xv[a:b], wv[e])
        ref.close(got[a:b], y, ref.rounded(y, err, F32), f"expert {e}")


# ----------------------------------------------- scale bytes over their range ----

# Rows of x for every kernel of the products: one row, few, K splits and tiles.
@pytest.mark.parametrize("M", [1, 20, 64, 300])
@pytest.mark.parametrize("low", [True, False], ids=["low-scales", "high-scales"])
def test_linear_every_scale(M, low):
    """Scale bytes 0 to 126 (2^-127 up: bf16 subnormals among the weights) with x about 2^90, 126 to 252 with
    x about 2^-100: every product is a normal float32."""
    K, N = 1056, 1024
    g = gen(M)
    x = (torch.randn(M, K, generator=g) * 2.0 ** (90 if low else -100)).to(BF16).cuda()
    w, s = matrix(5, N, K)
    each = torch.arange(N) % 127 + (0 if low else 126)
    s.copy_(each[:, None].expand(N, K // 32).to(torch.uint8))
    say("every scale", M, low)
    got = swq.mx4_linear(x, w, s, out_mode=swq.SWQ_LINEAR_F32)
    y, err = ref.dot(ref.to64(x), ref.values(w, s))
    ref.close(got, y, ref.rounded(y, err, F32), "every scale")


@pytest.mark.parametrize("M,N", [(20, 300), (70, 4096), (1500, 1544)])
def test_matmul_every_scale(M, N):
    """Scale bytes over their whole range on both sides, such that every product is a normal float32."""
    K = 96
    (a, sa), (w, s) = matrix(1, M, K), matrix(2, N, K)
    shift = torch.arange(N) % 251                                     # 2 .. 252 against 252 .. 2
    for lo in (2, 127, 252):
        sa.fill_(lo)
        s.copy_(torch.clamp(shift + 2, max=(127 + 127 + 100) - lo, min=max(2, 127 + 127 - 100 - lo))[:, None]
                .expand(N, K // 32).to(torch.uint8))
        say("matmul every scale", M, N, lo)
        got = swq.mx4_matmul(a, sa, w, s, out_mode=swq.SWQ_LINEAR_F32)
        y, err = ref.dot(ref.values(a, sa), ref.values(w, s))
        ref.close(got, y, ref.rounded(y, err, F32), f"matmul every scale {lo}")


@pytest.mark.parametrize("M,N", [(20, 300), (70, 4096), (1500, 1544), (3100, 3336)])
def test_matmul_nan_scales(M, N):
    """A NaN scale of either operand makes its row or its column NaN, and nothing else."""
    K = 160
    (a, sa), (w, s) = matrix(1, M, K), matrix(2, N, K)
    clean = swq.mx4_matmul(a, sa, w, s)
    sa[7, 1], s[N - 3, 4] = 255, 255
    say("matmul nan scales", M, N)
    got = swq.mx4_matmul(a, sa, w, s)
    bad = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    bad[7], bad[:, N - 3] = True, True
    assert torch.equal(torch.isnan(got), bad) and torch.equal(got[~bad], clean[~bad])


# ------------------------------------------------------ workspaces and graphs ----

@pytest.mark.parametrize("dtype", [BF16, F16])
def test_workspace_grows_after_a_capture(dtype):
    """Calls captured while the stream had a small workspace keep their results when an eager call of the
    same stream has made it larger, and when other calls use the larger one between the replays."""
    st = torch.cuda.Stream()
    x, (w, s) = acts(1, 64, 2080, dtype=dtype), matrix(2, 1024, 2080)
    xm, ids, weights, ws = moe_case(3, 40, 2, 4, 96, 64, 80, dtype)
    calls = lambda: [swq.mx4_linear(x, w, s), swq.moe_mlp(xm, ids, weights, *ws[0], *ws[1], *ws[2])]
    xl, il, wl, wsl = moe_case(5, 1500, 3, 5, 64, 1024, 520, dtype)
    large = lambda: swq.moe_mlp(xl, il, wl, *wsl[0], *wsl[1], *wsl[2])
    say("workspace grows after a capture", dtype)
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        want = [t.clone() for t in calls()]
    st.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        got = calls()
    with torch.cuda.stream(st):
        first = large().clone()
    st.synchronize()
    for rep in range(3):
        for t in got:
            t.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            again = large()
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(again, first)
        for p, q in zip(want, got):
            assert torch.equal(p, q), rep


# ----------------------------------------------------------------- LDS poison ----

@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("M,K,N", SPLIT)
def test_poison_k_split(poison, M, K, N, dtype):  # noqa: F811
    x, (w, s) = acts(M, M, K, dtype=dtype), matrix(N, N, K)
    say("poison k split", M, K, N, dtype)
    both(poison, lambda: swq.mx4_linear(x, w, s))


@pytest.mark.parametrize("P,E,kind", [(50, 66, "gaps"), (1000, 66, "unordered"), (4000, 130, "outside"),
                                      (5000, 1024, "covering")])
def test_poison_plan(poison, P, E, kind):  # noqa: F811
    """The plan from offsets, and from ids in one block and in eight."""
    x, (w, s), off = acts(P, P, 96), matrix(E, E, 70, 96), offsets_of(kind, P, E).cuda()
    say("poison plan", P, E, kind)
    both(poison, lambda: swq.mx4_grouped_linear(x, off, w, s))
    xm, ids, weights, ws = moe_case(P, P // 2, 2, E, 64, 32, 40, BF16)
    both(poison, lambda: swq.moe_mlp(xm, ids, weights, *ws[0], *ws[1], *ws[2]))
