"""The MXFP4 operators, the router and the experts' MLP on the GPU where a
caller's state or a size is out of the ordinary: errors that other code left
behind, operands of 4 GiB and more, more threads than one launch holds."""
import pytest
import torch

import mx4_reference as ref
import quantized_swiglu_forward_amd as swq
from gpu_helpers import say
from test_gpu_mx4 import BF16, F16, F32, HIDDEN, MODE, acts, matrix, moe_case

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _device():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    swq.lib()
    yield
    torch.cuda.synchronize()


def leave_an_error():
    """What a failed HIP call of other code leaves in this thread (the host refuses the device number)."""
    assert swq.lib().hipSetDevice(1 << 20) != 0


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("M", [1, 20, 300])
def test_error_of_other_code(M, dtype):
    """An error that an earlier call of other code left is not this call's: it runs and reports success."""
    t = swq.SWQ_TYPE_F16 if dtype == F16 else swq.SWQ_TYPE_BF16
    K, N, T, k, E = 96, 130, M, 2, 3
    x, (w, s) = acts(M, M, K, dtype=dtype), matrix(2, E, N, K)
    (wu, su), (wd, sd) = matrix(3, E, N // 32 * 32, K), matrix(4, E, K, N // 32 * 32)
    off = torch.tensor([0, M // 3, M // 2, M], dtype=torch.int32).cuda()
    _, ids, weights, _ = moe_case(1, T, k, E, 32, 32, 32, dtype)
    a, sa = swq.mx4_quantize(x)
    gate = w[:, :wu.shape[1]].contiguous(), s[:, :wu.shape[1]].contiguous()
    say("error of other code", M, dtype)
    want = [swq.mx4_linear(x, w[0], s[0]), swq.mx4_matmul(a, sa, w[0], s[0], out_mode=t),
            swq.mx4_grouped_linear(x, off, w, s), swq.moe_mlp(x, ids, weights, *gate, wu, su, wd, sd)]
    got = [torch.full_like(y, float("nan")) for y in want]
    torch.cuda.synchronize()
    calls = [lambda o: swq.swiglu_q_mx4_linear(x, w[0], s[0], None, M, K, N, t, t, o),
             lambda o: swq.swiglu_q_mx4_matmul(a, sa, w[0], s[0], M, K, N, t, o),
             lambda o: swq.swiglu_q_mx4_grouped_linear(x, off, w, s, M, E, K, N, t, t, o),
             lambda o: swq.swiglu_q_moe_mlp(x, ids, weights, *gate, wu, su, wd, sd, None, T, k, E, K, wu.shape[1], K,
                                            t, t, o)]
    for call, o in zip(calls, got):
        leave_an_error()
        assert call(o) == swq.SWQ_OK
    for p, q in zip(want, got):
        assert torch.equal(p, q)


# One operand of more than 4 GiB, whose rows come in two slabs (the second begins at 524544):
# rows of outputs of both widths, and as many outputs as the kernel for few could not launch.
PAST_4_GIB = [(1048876, 8192, 70), (1048876, 8192, 4096), (70, 8192, 1048877), (5, 8192, 1048880)]


@pytest.mark.parametrize("M,K,N", PAST_4_GIB)
def test_matmul_past_4_gib(M, K, N):
    rows = max(M, N)
    large = torch.zeros(rows, K // 8, dtype=torch.int32, device="cuda")
    scales = torch.full((rows, K // 32), 127, dtype=torch.uint8, device="cuda")
    pick = torch.tensor([0, 1, 300, rows // 3, 524543, 524544, 524671, 524672, 524700, rows - 2, rows - 1]).cuda()
    large[pick], scales[pick] = matrix(1, len(pick), K, lo=120, hi=134)
    c, s = matrix(2, min(M, N), K)
    for out in (BF16, F32) if M * N < 1 << 30 else (BF16,):
        say("matmul past 4 GiB", M, K, N, out)
        a, w = ((large, scales), (c, s)) if M > N else ((c, s), (large, scales))
        got = swq.mx4_matmul(*a, *w, out_mode=MODE[out])
        y, err = ref.dot(ref.values(large[pick], scales[pick]), ref.values(c, s))
        rows_of = got if M > N else got.t()
        ref.close(rows_of[pick], y, ref.rounded(y, err, out), f"past 4 GiB {out}")
        live = torch.zeros(rows, dtype=torch.bool, device="cuda")
        live[pick] = True
        assert torch.equal((rows_of != 0).any(1), live)          # (zero codes: zeros)


def room(gib):
    """Whether the card has this much memory left for a test; what torch holds unused is given back first."""
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gib << 30:
        pytest.skip(f"needs {gib} GiB of GPU memory")


def test_quantize_past_a_launch():
    """More than 2^35 elements, 2^32 words of codes: rows at the borders of the launches and the last ones
    against the same rows alone."""
    room(100)
    K = 1 << 17
    R = (1 << 18) + 3                                  # one launch takes 2^33 elements, 2^16 rows
    pick = [0, 1, 65535, 65536, 131071, 131072, 196608, 262143, 262144, R - 1]
    say("quantize past a launch")
    x = torch.zeros(R, K, dtype=BF16, device="cuda")
    part = acts(5, len(pick), K)
    x[pick] = part
    codes, scales = swq.mx4_quantize(x)
    c, s = swq.mx4_quantize(part)
    assert torch.equal(codes[pick], c) and torch.equal(scales[pick], s)
    live = torch.zeros(R, dtype=torch.bool, device="cuda")
    live[pick] = True
    rows_with = lambda t: torch.cat([(u != 0).any(1) for u in t.split(1 << 14)])
    assert torch.equal(rows_with(codes), live) and torch.equal(rows_with(scales), live)
    x.fill_(float("nan"))
    swq.mx4_dequantize(codes, scales, BF16, out=x)
    assert torch.equal(x[pick], swq.mx4_dequantize(c, s, BF16)) and torch.equal(rows_with(x), live)
    del x, codes, scales
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype,T,E", [(BF16, (1 << 28) + 5, 4), (F16, (1 << 24) + 3, 264), (F32, (1 << 24) + 3, 257)])
def test_route_past_a_launch(dtype, T, E):
    """Tokens of several launches (the first case: 2^32 threads in all and more): those at the borders and the last ones
    against the same tokens alone."""
    room(40)
    pick = torch.tensor([0, 1, (1 << 24) - 1, 1 << 24, T // 2, T - 2, T - 1]).cuda()
    lo = torch.zeros(T, E, dtype=dtype, device="cuda")
    lo[pick] = part = acts(3, len(pick), E, dtype=dtype)
    say("route past a launch", dtype, T, E)
    ids = torch.full((T, 2), -7, dtype=torch.int32, device="cuda")
    weights = torch.full((T, 2), float("nan"), device="cuda")
    swq.route(lo, 2, swq.SWQ_ROUTE_SOFTMAX_CHOSEN, ids=ids, weights=weights)
    i, w = swq.route(part, 2, swq.SWQ_ROUTE_SOFTMAX_CHOSEN)
    assert torch.equal(ids[pick], i) and torch.equal(weights[pick], w)
    ids[pick], weights[pick] = torch.tensor([0, 1], dtype=torch.int32, device="cuda"), 0.5
    assert bool((ids[:, 0] == 0).all()) and bool((ids[:, 1] == 1).all()) and bool((weights == 0.5).all())
    del lo, ids, weights
    torch.cuda.empty_cache()


@pytest.mark.parametrize("Ho", [257, 260])
def test_moe_sums_past_a_launch(Ho):
    """So many tokens that the sums over their experts take several launches, one output or four a thread:
    tokens at the borders (every 2^22nd, 2^24th) and the last ones against the formula."""
    room(80)
    T, H, I, E = (1 << 24) + 5, 32, 32, 2
    pick = torch.tensor([0, (1 << 22) - 1, 1 << 22, 3 << 22, (1 << 24) - 1, 1 << 24, T - 2, T - 1]).cuda()
    x = torch.zeros(T, H, dtype=BF16, device="cuda")
    x[pick] = acts(1, len(pick), H)
    ids = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
    ids[pick[1::2]] = 1
    weights = torch.full((T, 1), 0.75, device="cuda")
    ws = [matrix(2 + i, *sh) for i, sh in enumerate(((E, I, H), (E, I, H), (E, Ho, I)))]
    out = torch.full((T, Ho), float("nan"), dtype=BF16, device="cuda")
    say("moe sums past a launch", Ho)
    swq.moe_mlp(x, ids, weights, *ws[0], *ws[1], *ws[2], out=out)
    y, err = ref.experts(ref.to64(x[pick]), ids[pick].cpu().numpy(), ref.to64(weights[pick]),
                         *(ref.values(*w) for w in ws), None, HIDDEN[BF16])
    ref.close(out[pick], y, ref.rounded(y, err, BF16), "moe sums past a launch")
    out[pick] = 0
    assert not any(bool((part != 0).any()) for part in out.split(1 << 22))       # (zero rows: zeros)
    del x, out
    swq.swiglu_q_release_workspace()
    torch.cuda.empty_cache()


def test_linear_split_past_a_launch():
    """float16 rows of more than 2^33 elements, whose split takes several launches."""
    room(80)
    M, K, N = 8200, 1 << 20, 8
    pick = torch.tensor([0, 8191, 8192, M - 1]).cuda()
    x = torch.zeros(M, K, dtype=F16, device="cuda")
    x[pick] = acts(1, len(pick), K, dtype=F16)
    w, s = matrix(2, N, K)
    say("linear split past a launch")
    got = swq.mx4_linear(x, w, s, out_mode=swq.SWQ_LINEAR_F32)
    y, err = ref.dot(ref.to64(x[pick]), ref.values(w, s))
    ref.close(got[pick], y, ref.rounded(y, err, F32), "linear split past a launch")
    got[pick] = 0
    assert not bool(got.any())
    del x
    swq.swiglu_q_release_workspace()
    torch.cuda.empty_cache()
