"""The MXFP4 operators, the router and the experts' MLP on the GPU against
their plain 64-bit forms (mx4_reference), within the bounds derived there."""
import numpy as np
import pytest
import torch

import mx4_reference as ref
import quantized_swiglu_forward_amd as swq
from gpu_helpers import say

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
MODE = {BF16: swq.SWQ_LINEAR_BF16, F16: swq.SWQ_LINEAR_F16, F32: swq.SWQ_LINEAR_F32}
HIDDEN = {BF16: 2.0 ** -8, F16: 2.0 ** -16}


@pytest.fixture(autouse=True, scope="module")
def _device():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    swq.lib()
    yield
    torch.cuda.synchronize()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def matrix(seed, *shape, lo=119, hi=126):
    """Random codes and scales of values [*shape] on the GPU."""
    g = gen(seed)
    codes = torch.randint(-2 ** 31, 2 ** 31, (*shape[:-1], shape[-1] // 8), generator=g).to(torch.int32)
    scales = torch.randint(lo, hi, (*shape[:-1], shape[-1] // 32), generator=g).to(torch.uint8)
    return codes.cuda(), scales.cuda()


def acts(seed, *shape, dtype=BF16):
    return torch.randn(*shape, generator=gen(seed)).to(dtype).cuda()


# ---------------------------------------------------------------- quantise ----

@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("R,K", [(1, 32), (3, 96), (7, 2048), (65, 1056), (130, 64)])
def test_quantize(R, K, dtype):
    say("quantize", R, K, dtype)
    x = torch.randn(R, K, generator=gen(R + K)) * torch.exp2(torch.randint(-12, 12, (R, 1), generator=gen(K)).float())
    x = x.to(dtype).cuda()
    codes, scales = swq.mx4_quantize(x)
    qc, qs = ref.quantize(x)
    assert np.array_equal(ref.unpack(codes), qc) and np.array_equal(scales.cpu().numpy(), qs)
    for out in (BF16, F16, F32):
        v = swq.mx4_dequantize(codes, scales, out)
        y = ref.values(codes, scales)
        ref.close(v, y, ref.rounded(y, 0 * y, out) if out == F16 else 0 * y, f"dequantize {out}")


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_quantize_borders(dtype):
    """Every tie, saturation, zeros of both signs, the type's smallest and
    largest values, blocks with an infinity or a NaN, a whole row of zeros."""
    fi = torch.finfo(dtype)
    ties = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 4.0]
    rows = []
    for e in (-8, 0, 3):
        rows.append([v * 2.0 ** e for v in ties] + [-v * 2.0 ** e for v in ties] + [0.0, -0.0] * 6)
    rows.append([fi.max, -fi.max, fi.tiny, 0.0] * 8)
    rows.append([fi.tiny, fi.smallest_normal / 2, -fi.tiny, 0.0] * 8)
    rows.append([fi.smallest_normal * fi.eps, 0.0] * 16)                 # subnormals alone
    rows.append([float("inf")] + [1.0] * 31)
    rows.append([1.0] * 31 + [float("nan")])
    rows.append([0.0, -0.0] * 16)
    x = torch.tensor(rows, dtype=torch.float64).to(dtype).cuda()
    say("quantize borders", dtype)
    codes, scales = swq.mx4_quantize(x)
    qc, qs = ref.quantize(x)
    assert np.array_equal(scales.cpu().numpy(), qs)
    assert np.array_equal(ref.unpack(codes), qc)
    v = swq.mx4_dequantize(codes, scales, F32).cpu()
    assert torch.isnan(v[6:8]).all() and not torch.isnan(v[:6]).any()


def test_dequantize_every_scale():
    """All 256 scale bytes against all 16 codes, in each type."""
    codes = torch.tensor([0x76543210, -0x01234568, 0, 0], dtype=torch.int32).repeat(256, 1).cuda()
    scales = torch.arange(256).to(torch.uint8)[:, None].cuda()
    say("dequantize every scale")
    y = ref.values(codes, scales)
    for dtype in (F32, BF16, F16):
        v = swq.mx4_dequantize(codes, scales, dtype).cpu()
        assert torch.equal(torch.nan_to_num(v, nan=-1.0, posinf=-2.0, neginf=-3.0),
                           torch.nan_to_num(torch.from_numpy(y).to(dtype), nan=-1.0, posinf=-2.0, neginf=-3.0)), dtype


def test_quantize_past_32_bits():
    """More than 2^32 elements: the last rows against the same rows alone."""
    R, K = 1 << 17, 32 * 1031
    say("quantize past 32 bits")
    x = torch.zeros(R, K, dtype=BF16, device="cuda")
    tail = acts(5, 3, K)
    x[-3:] = tail
    codes, scales = swq.mx4_quantize(x)
    c, s = swq.mx4_quantize(tail)
    assert torch.equal(codes[-3:], c) and torch.equal(scales[-3:], s) and not codes[:-3].any()
    out = swq.mx4_dequantize(codes, scales, BF16)
    assert torch.equal(out[-3:], swq.mx4_dequantize(c, s, BF16)) and not out[:-3].any()


# ---------------------------------------------------------------- products ----

LINEAR = [(1, 32, 1), (1, 2048, 300), (2, 96, 17), (3, 4096, 33), (5, 5632, 129), (15, 160, 16), (16, 512, 100),
          (17, 1056, 257), (31, 2080, 64), (33, 64, 130), (64, 1024, 515), (65, 352, 128), (100, 2048, 31),
          (129, 256, 640), (200, 992, 1001), (257, 1536, 259), (300, 128, 300), (513, 608, 770)]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("M,K,N", LINEAR)
def test_linear(M, K, N, dtype):
    x, (w, s) = acts(M + N, M, K, dtype=dtype), matrix(K + N, N, K)
    res = acts(N, M, N, dtype=dtype)
    y, err = ref.dot(ref.to64(x), ref.values(w, s))
    for out, r in ((dtype, None), (F32, None), (dtype, res), (F32, res)):
        say("linear", M, K, N, dtype, "out", out, "residual", r is not None)
        got = swq.mx4_linear(x, w, s, residual=r, out_mode=MODE[out])
        yy, ee = (y, err) if r is None else (y + ref.to64(r), err + 2.0 ** -23 * (np.abs(y) + np.abs(ref.to64(r))))
        ref.close(got, yy, ref.rounded(yy, ee, out), f"linear M{M} K{K} N{N} {out}")


@pytest.mark.parametrize("M,K,N", LINEAR)
def test_matmul(M, K, N):
    (a, sa), (w, s) = matrix(M + 1, M, K, lo=120, hi=134), matrix(K + N, N, K)
    y, err = ref.dot(ref.values(a, sa), ref.values(w, s))
    for out in (BF16, F16, F32):
        say("matmul", M, K, N, out)
        got = swq.mx4_matmul(a, sa, w, s, out_mode=MODE[out])
        ref.close(got, y, ref.rounded(y, err, out), f"matmul M{M} K{K} N{N} {out}")


# (M, K, N) that take the 128 x 128 and the 128 x 256 tiles: aligned rows, rows of 4, odd rows
@pytest.mark.parametrize("M,K,N", [(513, 160, 5700), (600, 96, 5632), (2047, 288, 4090), (1900, 544, 4096)])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_linear_large_tiles(M, K, N, dtype):
    x, (w, s) = acts(M, M, K, dtype=dtype), matrix(N, N, K)
    res = acts(N, M, N, dtype=dtype)
    y, err = ref.dot(ref.to64(x), ref.values(w, s))
    for out, r in ((dtype, res), (F32, None)):
        say("linear large", M, K, N, dtype, out)
        got = swq.mx4_linear(x, w, s, residual=r, out_mode=MODE[out])
        yy, ee = (y, err) if r is None else (y + ref.to64(r), err + 2.0 ** -23 * (np.abs(y) + np.abs(ref.to64(r))))
        ref.close(got, yy, ref.rounded(yy, ee, out), f"linear large {out}")


# the 128 x 128 and the 256 x 256 tiles of two MXFP4 operands
@pytest.mark.parametrize("M,K,N", [(1500, 160, 1530), (1500, 1056, 1544), (3100, 288, 3300), (3100, 416, 3336)])
def test_matmul_large_tiles(M, K, N):
    (a, sa), (w, s) = matrix(M + 1, M, K, lo=120, hi=134), matrix(K + N, N, K)
    y, err = ref.dot(ref.values(a, sa), ref.values(w, s))
    for out in (BF16, F16, F32):
        say("matmul large", M, K, N, out)
        got = swq.mx4_matmul(a, sa, w, s, out_mode=MODE[out])
        ref.close(got, y, ref.rounded(y, err, out), f"matmul large {out}")


# their 64 x 64 tiles: more 16 x 16 tiles than the kernel for few outputs takes
@pytest.mark.parametrize("M,K,N", [(500, 160, 1030), (531, 1056, 1000), (20, 416, 9004), (300, 2080, 1001)])
def test_matmul_small_tiles(M, K, N):
    (a, sa), (w, s) = matrix(M + 1, M, K, lo=120, hi=134), matrix(K + N, N, K)
    y, err = ref.dot(ref.values(a, sa), ref.values(w, s))
    for out in (BF16, F16, F32):
        say("matmul small tiles", M, K, N, out)
        got = swq.mx4_matmul(a, sa, w, s, out_mode=MODE[out])
        ref.close(got, y, ref.rounded(y, err, out), f"matmul small tiles {out}")


def test_leading_dimensions_and_empty():
    x, (w, s) = acts(1, 2, 3, 64), matrix(2, 40, 64)
    say("leading dimensions")
    y = swq.mx4_linear(x, w, s)
    assert y.shape == (2, 3, 40) and torch.equal(y.reshape(6, 40), swq.mx4_linear(x.reshape(6, 64), w, s))
    assert swq.mx4_linear(x[:0], w, s).shape == (0, 3, 40)
    c, cs = swq.mx4_quantize(x)
    assert c.shape == (2, 3, 8) and cs.shape == (2, 3, 2)
    assert swq.mx4_matmul(c, cs, w, s).shape == (2, 3, 40)
    assert swq.mx4_matmul(c[:0], cs[:0], w, s).shape == (0, 3, 40)
    assert swq.mx4_quantize(x[:0])[0].shape == (0, 3, 8)
    assert swq.mx4_dequantize(c[:0], cs[:0]).shape == (0, 3, 64)


@pytest.mark.parametrize("M", [1, 7, 40, 300])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_nonfinite_stays_in_its_row_and_column(M, dtype):
    """An infinity or a NaN in a row of x, a NaN scale in a row of W: that row
    and that column alone are affected."""
    K, N = 288, 150
    x, (w, s) = acts(3, M, K, dtype=dtype), matrix(4, N, K)
    s[77, 3] = 255
    if M > 2:
        x[1, 5], x[2, 200] = float("nan"), float("inf")
    say("nonfinite", M, dtype)
    y = swq.mx4_linear(x, w, s, out_mode=swq.SWQ_LINEAR_F32).cpu()
    clean_x, clean_s = x.clone(), s.clone()
    clean_s[77, 3] = 120
    if M > 2:
        clean_x[1:3] = 0
    z = swq.mx4_linear(clean_x, w, clean_s, out_mode=swq.SWQ_LINEAR_F32).cpu()
    rows = [m for m in range(M) if M <= 2 or m not in (1, 2)]
    cols = [n for n in range(N) if n != 77]
    assert torch.isnan(y[:, 77]).all()
    assert torch.equal(y[rows][:, cols], z[rows][:, cols])
    if M > 2:
        assert torch.isnan(y[1]).all() and not torch.isfinite(y[2]).any()


def test_scales_at_any_address():
    """Scales need no alignment: a view that starts at an odd byte."""
    x, (w, s) = acts(1, 20, 352), matrix(2, 200, 352)
    raw = torch.empty(s.numel() + 3, dtype=torch.uint8, device="cuda")
    odd = raw[3:].view(s.shape)
    odd.copy_(s)
    say("odd scale address")
    for m in (1, 20):
        assert torch.equal(swq.mx4_linear(x[:m], w, odd), swq.mx4_linear(x[:m], w, s))
    a, sa = swq.mx4_quantize(x)
    assert torch.equal(swq.mx4_matmul(a, sa, w, odd), swq.mx4_matmul(a, sa, w, s))


# ----------------------------------------------------------------- grouped ----

GROUPED = [([0, 5, 5, 6, 40], 96, 33), ([0, 0, 0, 1], 2048, 130), ([0, 17, 300, 300, 310], 352, 257),
           ([0, 1, 2, 3, 4, 5, 6, 7, 8], 64, 100), ([0, 260, 520], 544, 300), ([0, 3], 160, 5)]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("offsets,K,N", GROUPED, ids=[f"E{len(g[0]) - 1}-P{g[0][-1]}" for g in GROUPED])
def test_grouped(offsets, K, N, dtype):
    P, E = offsets[-1], len(offsets) - 1
    x, (w, s) = acts(P, P, K, dtype=dtype), matrix(K, E, N, K)
    off = torch.tensor(offsets, dtype=torch.int32).cuda()
    wv = ref.values(w, s)
    parts = [ref.dot(ref.to64(x[a:b]), wv[e]) for e, (a, b) in enumerate(zip(offsets, offsets[1:]))]
    y, err = (np.concatenate([p[i] for p in parts]) for i in (0, 1))
    for out in (dtype, F32):
        say("grouped", offsets, K, N, dtype, out)
        got = swq.mx4_grouped_linear(x, off, w, s, out_mode=MODE[out])
        ref.close(got, y, ref.rounded(y, err, out), f"grouped {offsets} {out}")


@pytest.mark.parametrize("P", [12, 400])
@pytest.mark.parametrize("offsets,taken", [([2, 5, 9], [2, 5, 9]), ([-3, 4, 10 ** 9], [0, 4, None]),
                                           ([0, 8, 3], [0, 8, 8]), ([9, 9, 9], [9, 9, 9])])
def test_grouped_odd_offsets(P, offsets, taken):
    """Rows of no group are zero; offsets that decrease or leave the rows are
    taken as the nearest that do not."""
    x, (w, s) = acts(1, P, 96), matrix(2, 2, 70, 96)
    taken = [P if t is None else t for t in taken]
    out = torch.full((P, 70), float("nan"), dtype=BF16, device="cuda")
    say("grouped odd offsets", P, offsets)
    swq.mx4_grouped_linear(x, torch.tensor(offsets, dtype=torch.int32).cuda(), w, s, out=out)
    want = torch.zeros_like(out)
    for e in range(2):
        a, b = taken[e], taken[e + 1]
        if b > a:
            want[a:b] = swq.mx4_linear(x[a:b].contiguous(), w[e], s[e])
    assert torch.equal(out == 0, want == 0) and not torch.isnan(out).any()
    y = ref.values(w, s)
    for e in range(2):
        a, b = taken[e], taken[e + 1]
        if b > a:
            v, err = ref.dot(ref.to64(x[a:b]), y[e])
            ref.close(out[a:b], v, ref.rounded(v, err, BF16), "odd offsets")


def test_most_experts():
    """1024 experts, most of them without a row, the first and the last with some."""
    E, N, K, P = 1024, 40, 64, 50
    w, s = matrix(3, E, N, K)
    expert = torch.cat([torch.zeros(3, dtype=torch.long), torch.randint(0, E, (P - 7,), generator=gen(1)),
                        torch.full((4,), E - 1)]).sort().values
    off = torch.searchsorted(expert, torch.arange(E + 1)).to(torch.int32)
    x = acts(2, P, K)
    say("most experts")
    got = swq.mx4_grouped_linear(x, off.cuda(), w, s, out_mode=swq.SWQ_LINEAR_F32)
    wv = ref.values(w, s)
    y, err = (np.concatenate([ref.dot(ref.to64(x[p:p + 1]), wv[int(expert[p])])[i] for p in range(P)]) for i in (0, 1))
    ref.close(got, y, ref.rounded(y, err, F32), "most experts")
    wd, sd = matrix(4, E, 48, 32)
    h = [matrix(5 + i, E, 32, K) for i in (0, 1)]
    ids = torch.stack([expert[torch.randperm(P, generator=gen(9))], expert], 1).to(torch.int32).cuda()
    weights = torch.rand(P, 2, generator=gen(8)).cuda()
    got = swq.moe_mlp(x, ids, weights, *h[0], *h[1], wd, sd)
    y, err = ref.experts(ref.to64(x), ids.cpu().numpy(), ref.to64(weights), ref.values(*h[0]), ref.values(*h[1]),
                         ref.values(wd, sd), None, HIDDEN[BF16])
    ref.close(got, y, ref.rounded(y, err, BF16), "most experts, MLP")


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("T,E,k,H,I,Ho", [(700, 3, 1, 64, 4096, 40), (700, 3, 1, 2048, 32, 4100), (400, 2, 2, 96, 96, 2052),
                                            (10300, 3, 2, 64, 32, 2056), (20500, 2, 1, 32, 32, 2050)])
def test_moe_unlike_widths(T, E, k, H, I, Ho, dtype):
    """Wide and narrow hidden tensors, where both products take the tiles of one plan, and outputs so large
    that they are computed and summed some columns at a time."""
    x, ids, weights, ((wg, sg), (wu, su), (wd, sd)) = moe_case(T + I, T, k, E, H, I, Ho, dtype)
    say("moe unlike widths", T, E, k, H, I, Ho, dtype)
    got = swq.moe_mlp(x, ids, weights, wg, sg, wu, su, wd, sd, out_mode=swq.SWQ_LINEAR_F32)
    pick = torch.cat([torch.arange(0, T, max(37, T // 30)), torch.tensor([T - 1])])
    y, err = ref.experts(ref.to64(x)[pick], ids.cpu().numpy()[pick], ref.to64(weights)[pick],
                         *(ref.values(w, s) for w, s in ((wg, sg), (wu, su), (wd, sd))), None, HIDDEN[dtype])
    ref.close(got[pick.cuda()], y, ref.rounded(y, err, F32), "moe unlike widths")


def test_grouped_weights_past_4_gib():
    """The last expert of a set of more than 2^32 bytes of codes."""
    E, N, K = 66, 16384, 8192
    say("grouped past 4 GiB")
    w = torch.zeros(E, N, K // 8, dtype=torch.int32, device="cuda")
    s = torch.full((E, N, K // 32), 127, dtype=torch.uint8, device="cuda")
    cw, cs = matrix(9, N, K)
    w[-1], s[-1] = cw, cs
    for rows in (3, 70):
        x = acts(rows, rows, K)
        off = torch.zeros(E + 1, dtype=torch.int32)
        off[-1] = rows
        got = swq.mx4_grouped_linear(x, off.cuda(), w, s, out_mode=swq.SWQ_LINEAR_F32)
        n = torch.arange(0, N, 511)
        y, err = ref.dot(ref.to64(x), ref.values(cw[n.cuda()], cs[n.cuda()]))
        ref.close(got[:, n.cuda()], y, ref.rounded(y, err, F32), "past 4 GiB")


# ------------------------------------------------------------------ router ----

ROUTE_TOL = 64 * 2.0 ** -24     # exp and its sum over up to 1024 terms: a few units each, and the quotient


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 64, 4), (5, 7, 7), (33, 128, 8), (200, 256, 8), (64, 1000, 20),
                                   (3, 1024, 64), (70, 60, 6), (17, 512, 10), (9, 33, 2)])
def test_route(T, E, k, dtype):
    lo = (2 * torch.randn(T, E, generator=gen(T + E))).to(dtype)
    if dtype != F32:
        lo[:, E // 2:] = lo[:, :E - E // 2]              # equal logits: the lower index wins
    for scoring in range(4):
        say("route", T, E, k, dtype, scoring)
        ids, w = swq.route(lo.cuda(), k, scoring)
        ri, rw = ref.route(lo, k, scoring)
        assert np.array_equal(ids.cpu().numpy(), ri)
        # a sum of n terms: n units of 2^-24 at most
        assert np.all(np.abs(ref.to64(w) - rw) <= (ROUTE_TOL + E * 2.0 ** -24) * rw + 2.0 ** -149)


def test_route_masks_and_nonfinite():
    """Rows with fewer than k experts left, with none, with NaN, with +inf, with
    all logits equal, with the type's lowest value as a mask."""
    inf, nan = float("inf"), float("nan")
    low = torch.finfo(F32).min
    lo = torch.tensor([[-inf, 1.0, -inf, -inf, -inf], [-inf] * 5, [nan, 2.0, nan, 1.0, 3.0], [0.0, inf, 1.0, inf, -1.0],
                       [0.5] * 5, [low, low, 1.0, low, low], [nan] * 5, [low] * 5, [-0.0, 0.0, -0.0, 0.0, 0.0],
                       [-200.0, -300.0, -400.0, -inf, -1000.0], [inf, -low, inf, -low, 0.0], [-inf, nan, inf, nan, -inf]])
    for scoring in range(4):
        say("route masks", scoring)
        ids, w = swq.route(lo.cuda(), 3, scoring)
        ri, rw = ref.route(lo, 3, scoring)
        assert np.array_equal(ids.cpu().numpy(), ri), (scoring, ids.tolist(), ri.tolist())
        assert not torch.isnan(w).any()
        got = ref.to64(w)
        assert np.all(np.abs(got - rw) <= ROUTE_TOL * rw + 2.0 ** -126), (scoring, got.tolist(), rw.tolist())


# ----------------------------------------------------------------- experts ----

def moe_case(seed, T, k, E, H, I, Ho, dtype, spread=True):
    g = gen(seed)
    x = acts(seed, T, H, dtype=dtype)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32)
    if spread and T > 2:
        ids[0] = -1                                       # a token of no expert
        ids[1, k // 2] = E                                # an id past the experts
    weights = torch.rand(T, k, generator=g)
    ws = [matrix(seed + i, *sh) for i, sh in enumerate(((E, I, H), (E, I, H), (E, Ho, I)))]
    return x, ids.cuda(), weights.cuda(), ws


MOE = [(1, 2, 4, 64, 32, 64), (1, 8, 16, 2048, 96, 130), (3, 1, 2, 96, 64, 33), (5, 4, 8, 160, 224, 96),
       (20, 6, 6, 128, 352, 257), (40, 8, 60, 256, 160, 128), (130, 2, 3, 512, 96, 200), (300, 3, 5, 96, 288, 64),
       (70, 1, 1, 64, 64, 64), (1500, 3, 5, 64, 32, 64), (1100, 4, 37, 64, 96, 40)]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("T,k,E,H,I,Ho", MOE)
def test_moe_mlp(T, k, E, H, I, Ho, dtype):
    x, ids, weights, ((wg, sg), (wu, su), (wd, sd)) = moe_case(T + E, T, k, E, H, I, Ho, dtype)
    res = acts(7, T, Ho, dtype=dtype)
    v = [ref.values(w, s) for w, s in ((wg, sg), (wu, su), (wd, sd))]
    for r, out in ((None, dtype), (res, dtype), (res, F32)):
        say("moe", T, k, E, H, I, Ho, dtype, out, "residual", r is not None)
        got = swq.moe_mlp(x, ids, weights, wg, sg, wu, su, wd, sd, residual=r, out_mode=MODE[out])
        y, err = ref.experts(ref.to64(x), ids.cpu().numpy(), ref.to64(weights), *v,
                             None if r is None else ref.to64(r), HIDDEN[dtype])
        ref.close(got, y, ref.rounded(y, err, out), f"moe T{T} k{k} E{E} {out}")


@pytest.mark.parametrize("T", [1, 4, 100])
def test_moe_skipped_slots(T):
    """Tokens with no expert give the residual; a NaN weight or a NaN row of
    weights of a skipped slot or an unused expert reaches nothing."""
    x, ids, weights, ((wg, sg), (wu, su), (wd, sd)) = moe_case(11, T, 2, 3, 64, 32, 64, BF16, spread=False)
    res = acts(1, T, 64)
    ids[:] = 1
    ids[:, 1] = -1
    weights[:, 1] = float("nan")
    sg[0], su[2], sd[0] = 255, 255, 255
    say("moe skipped", T)
    y = swq.moe_mlp(x, ids, weights, wg, sg, wu, su, wd, sd, residual=res)
    one = swq.moe_mlp(x, ids[:, :1].contiguous(), weights[:, :1].contiguous(), wg, sg, wu, su, wd, sd, residual=res)
    assert torch.equal(y, one) and not torch.isnan(y).any()
    ids[:] = -1
    assert torch.equal(swq.moe_mlp(x, ids, weights, wg, sg, wu, su, wd, sd, residual=res), res)
    assert not swq.moe_mlp(x, ids, weights, wg, sg, wu, su, wd, sd).any()


def test_routed_layer_end_to_end():
    """Quantiser, router and experts together: weights quantized from float32,
    logits through the router, its ids and weights into the experts' MLP."""
    T, E, k, H, I = 24, 8, 2, 128, 64
    x = acts(2, T, H)
    full = [torch.randn(E, n, m, generator=gen(30 + i)).cuda() * m ** -0.5 for i, (n, m) in
            enumerate(((I, H), (I, H), (H, I)))]
    q = [swq.mx4_quantize(w) for w in full]
    logits = torch.randn(T, E, generator=gen(4)).cuda()
    say("routed layer")
    ids, weights = swq.route(logits, k, swq.SWQ_ROUTE_SOFTMAX_CHOSEN)
    y = swq.moe_mlp(x, ids, weights, *q[0], *q[1], *q[2], residual=x)
    ri, rw = ref.route(logits, k, 1)
    assert np.array_equal(ids.cpu().numpy(), ri)
    v, err = ref.experts(ref.to64(x), ri, ref.to64(weights), *(ref.values(*t) for t in q), ref.to64(x), HIDDEN[BF16])
    ref.close(y, v, ref.rounded(v, err, BF16), "routed layer")


# ------------------------------------------------- streams, graphs, repeats ----

def _all_calls(seed, rows):
    x, ids, weights, ((wg, sg), (wu, su), (wd, sd)) = moe_case(seed, rows, 2, 4, 96, 64, 80, BF16)
    off = torch.tensor([0, rows // 3, rows // 3, rows - rows // 4, rows], dtype=torch.int32).cuda()
    lo = torch.randn(rows, 40, generator=gen(seed)).cuda()

    def run():
        c, s = swq.mx4_quantize(x)
        return [c, s, swq.mx4_dequantize(c, s), swq.mx4_linear(x, wg[0], sg[0]),
                swq.mx4_matmul(c, s, wg[1], sg[1], out_mode=swq.SWQ_LINEAR_F32),
                swq.mx4_grouped_linear(x, off, wu, su), *swq.route(lo, 5),
                swq.moe_mlp(x, ids, weights, wg, sg, wu, su, wd, sd)]
    return run


@pytest.mark.parametrize("rows", [1, 6, 150])
def test_repeats_and_other_stream(rows):
    """The same bits again, and on another stream."""
    run = _all_calls(rows, rows)
    say("repeats", rows)
    a = [t.clone() for t in run()]
    b = run()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        c = run()
    torch.cuda.current_stream().wait_stream(st)
    torch.cuda.synchronize()
    for p, q, r in zip(a, b, c):
        assert torch.equal(p, q) and torch.equal(p, r)


@pytest.mark.parametrize("rows", [1, 6, 150])
def test_graph_replays(rows):
    """Captured after one warm-up call, replayed with eager work between."""
    run, other = _all_calls(rows, rows), _all_calls(rows + 1, max(1, rows - 1))
    say("graph", rows)
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        want = [t.clone() for t in run()]
    st.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        got = run()
    for rep in range(3):
        for t in got:
            t.zero_()
        with torch.cuda.stream(st):
            other()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for p, q in zip(want, got):
            assert torch.equal(p, q), rep
