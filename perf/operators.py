"""Cases of the microscaled 4-bit (MXFP4) operators and of the experts' MLP:
what each computes in elementary torch operations, and the calls a user makes.

Formats: e2m1 codes, eight to a 32-bit word along K (code j in bits
[4j, 4j+4)), one e8m0 scale byte per 32 inputs.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
OUT_MODE = {torch.bfloat16: 0, torch.float32: 1, torch.float16: 2}    # the library's SWQ_LINEAR_BF16, _F32, _F16
SCORING = {"softmax": 0, "softmax_chosen": 1, "sigmoid": 2, "sigmoid_chosen": 3}    # its SWQ_ROUTE_* values
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
MX4_BYTES = 0.5 + 1.0 / 32.0     # of one element: its code and its share of a scale


def calls():
    import quantized_swiglu_forward_amd as swq
    return swq


# ------------------------------------------------------------------- cases ----

def listed():
    return [
        # one activation tile of a small batch quantized and read back
        {"name": "quantize-48x2048", "op": "quantize", "R": 48, "K": 2048, "type": "bf16"},
        # a long prefill's hidden tensor
        {"name": "quantize-8192x10240", "op": "quantize", "R": 8192, "K": 10240, "type": "bf16"},
        # decode: one token through a projection
        {"name": "linear-1x2048x5632", "op": "linear", "M": 1, "K": 2048, "N": 5632, "type": "bf16", "out": "bf16",
         "residual": False},
        # prefill: the large model's expansion
        {"name": "linear-2048x4096x14336", "op": "linear", "M": 2048, "K": 4096, "N": 14336, "type": "bf16",
         "out": "bf16", "residual": False},
        # both operands in 4 bits, a ragged middle-sized batch, float32 sums returned
        {"name": "matmul-200x2080x1001", "op": "matmul", "M": 200, "K": 2080, "N": 1001, "out": "f32"},
        # both operands in 4 bits, a long prefill
        {"name": "matmul-8192x2560x10240", "op": "matmul", "M": 8192, "K": 2560, "N": 10240, "out": "bf16"},
        # the router of one new token
        {"name": "route-1x64-top4", "op": "route", "T": 1, "E": 64, "k": 4, "type": "f32", "scoring": "softmax_chosen"},
        # the router of a long prefill, many experts
        {"name": "route-8192x256-top8", "op": "route", "T": 8192, "E": 256, "k": 8, "type": "bf16",
         "scoring": "softmax"},
        # decode: one token through its experts' MLPs
        {"name": "experts-1x64-top8", "op": "experts", "T": 1, "E": 64, "k": 8, "H": 2048, "I": 1024, "type": "bf16",
         "residual": True},
        # prefill through the experts
        {"name": "experts-4096x64-top8", "op": "experts", "T": 4096, "E": 64, "k": 8, "H": 2048, "I": 1024,
         "type": "bf16", "residual": True},
        # a decode batch's rows, already sorted by expert, float16
        {"name": "grouped-70x32x1504x2049", "op": "grouped", "P": 70, "E": 32, "K": 1504, "N": 2049, "type": "f16",
         "out": "f16", "skew": True},
        # a prefill's rows sorted by expert, uneven groups, some empty
        {"name": "grouped-6007x32x2048x1408", "op": "grouped", "P": 6007, "E": 32, "K": 2048, "N": 1408,
         "type": "bf16", "out": "bf16", "skew": True},
    ]


def _log(rng, lo, hi):
    """A size between lo and hi, even over its logarithm: an odd number (ragged tiles), four times one, or a power of two."""
    n = math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))
    form = rng.randrange(3)
    n = int(n) | 1 if form == 0 else 4 * (int(n / 4) | 1) if form == 1 and n >= 4 else 1 << int(round(math.log2(n)))
    return max(lo, min(hi, n))


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        b, f = most.get(c["op"], (0, 0))
        most[c["op"]] = (max(b, w["bytes"]), max(f, w["flops"]))
    while True:
        op = rng.choice(["quantize", "linear", "matmul", "route", "experts", "grouped"])
        if op == "quantize":
            c = {"R": _log(rng, 1, 16384), "K": 32 * _log(rng, 1, 448), "type": rng.choice(["bf16", "f16", "f32"])}
        elif op in ("linear", "matmul"):
            c = {"M": _log(rng, 1, 8192), "K": 32 * _log(rng, 2, 320), "N": _log(rng, 8, 14336)}
            if op == "linear":
                c["type"] = rng.choice(["bf16", "bf16", "f16"])
                c["out"] = rng.choice([c["type"], c["type"], "f32"])
                c["residual"] = rng.random() < 0.5
            else:
                c["out"] = rng.choice(["bf16", "f16", "f32"])
        elif op == "route":
            E = _log(rng, 4, 512)
            c = {"T": _log(rng, 1, 8192), "E": E, "k": rng.randint(1, min(10, E)),
                 "type": rng.choice(["bf16", "f16", "f32"]),
                 "scoring": rng.choice(["softmax", "softmax_chosen", "sigmoid", "sigmoid_chosen"])}
        elif op == "experts":
            E = _log(rng, 2, 64)
            c = {"T": _log(rng, 1, 4096), "E": E, "k": rng.randint(1, min(8, E)), "H": 32 * _log(rng, 4, 64),
                 "I": 32 * _log(rng, 3, 44), "type": rng.choice(["bf16", "bf16", "f16"]),
                 "residual": rng.random() < 0.5}
        else:
            t = rng.choice(["bf16", "bf16", "f16"])
            c = {"P": _log(rng, 1, 6007), "E": _log(rng, 2, 64), "K": 32 * _log(rng, 2, 88), "N": _log(rng, 8, 4096),
                 "type": t, "out": rng.choice([t, "f32"]), "skew": rng.random() < 0.5}
        c = {"op": op, **c}
        w = work(c)
        if w["bytes"] <= most[op][0] and w["flops"] <= most[op][1]:
            return c


def work(c):
    """Each input once, each output once; of the experts, as many as the rows can reach at most."""
    op = c["op"]
    if op == "quantize":        # in, codes and scales out; codes and scales in, values out
        n = c["R"] * c["K"]
        return {"bytes": n * 2 * (SIZE[c["type"]] + MX4_BYTES), "flops": 0}
    if op == "linear":
        M, K, N = c["M"], c["K"], c["N"]
        res = M * N * SIZE[c["type"]] if c["residual"] else 0
        return {"bytes": N * K * MX4_BYTES + M * K * SIZE[c["type"]] + M * N * SIZE[c["out"]] + res,
                "flops": 2 * M * N * K}
    if op == "matmul":
        M, K, N = c["M"], c["K"], c["N"]
        return {"bytes": (N + M) * K * MX4_BYTES + M * N * SIZE[c["out"]], "flops": 2 * M * N * K}
    if op == "route":
        return {"bytes": c["T"] * c["E"] * SIZE[c["type"]] + c["T"] * c["k"] * 8, "flops": 0}
    if op == "experts":
        T, k, H, I = c["T"], c["k"], c["H"], c["I"]
        act = min(c["E"], T * k)
        rows = T * H * SIZE[c["type"]]
        return {"bytes": act * 3 * H * I * MX4_BYTES + rows * (3 if c["residual"] else 2) + T * k * 8,
                "flops": 6 * T * k * H * I}
    P, K, N = c["P"], c["K"], c["N"]
    act = min(c["E"], P)
    return {"bytes": act * N * K * MX4_BYTES + P * K * SIZE[c["type"]] + P * N * SIZE[c["out"]], "flops": 2 * P * N * K}


# --------------------------------------------------------- elementary parts ----

def _e2m1(dtype, device):
    m = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=dtype, device=device)
    return torch.cat([m, -m])


def _quantize(x):
    """(codes int32 [..., K/8], scales uint8 [..., K/32]) in float32 steps."""
    K = x.shape[-1]
    b = x.float().reshape(-1, K // 32, 32)
    amax = b.abs().amax(-1)
    e = torch.frexp(amax).exponent - 3                      # floor(log2 amax) - 2
    e = torch.where(amax > 0, e, torch.full_like(e, -127)).clamp(-127, 127)
    fine = torch.isfinite(amax)
    e = torch.where(fine, e, torch.zeros_like(e))
    a = torch.ldexp(b.abs(), -e[..., None])
    q = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int()
         + (a >= 3.5).int() + (a > 5.0).int() + 8 * torch.signbit(b).int())
    q = torch.where(fine[..., None], q, torch.zeros_like(q)).reshape(-1, K // 8, 8)
    w = q[..., 0].clone()
    w |= (q[..., 1] << 4) | (q[..., 2] << 8) | (q[..., 3] << 12) | (q[..., 4] << 16) | (q[..., 5] << 20)
    w |= (q[..., 6] << 24) | (q[..., 7] << 28)
    s = torch.where(fine, e + 127, torch.full_like(e, 255)).to(torch.uint8)
    return w.reshape(*x.shape[:-1], K // 8), s.reshape(*x.shape[:-1], K // 32)


def _values(codes, scales, dtype=torch.float32):
    """The values [..., K] that codes and scales stand for."""
    sh = torch.arange(0, 32, 4, device=codes.device, dtype=torch.int32)
    q = (codes[..., None] >> sh) & 15
    v = _e2m1(dtype, codes.device)[q.long()].reshape(*scales.shape, 32)
    s = torch.exp2(scales.to(dtype) - 127.0)
    s = torch.where(scales == 255, torch.full_like(s, float("nan")), s)
    return (v * s[..., None]).reshape(*codes.shape[:-1], -1)


def _silu(t):
    return t / (1.0 + torch.exp(-t))


def _groups(expert, E):
    """Rows of each expert in a padded table: (row numbers [E, C], valid)."""
    counts = (expert[None, :] == torch.arange(E, device=expert.device)[:, None]).sum(1)
    order = torch.sort(expert, stable=True).indices
    first = torch.cumsum(counts, 0) - counts
    C = max(1, int(counts.max()))
    at = torch.arange(C, device=expert.device)
    valid = at[None, :] < counts[:, None]
    return order[torch.where(valid, first[:, None] + at[None, :], torch.zeros_like(at)[None, :])], valid


def _table(expert, E, few):
    """For few rows: a weight set per row instead of a table over all experts."""
    if few:
        n = torch.arange(expert.shape[0], device=expert.device)
        return n[:, None], torch.ones_like(n[:, None], dtype=torch.bool), expert
    rows, valid = _groups(expert, E)
    return rows, valid, slice(None)


def _scatter(y, rows, valid, P):
    out = torch.zeros(P, y.shape[-1], dtype=y.dtype, device=y.device)
    out[rows[valid]] = y[valid]
    return out


def _times(x, w):
    """x [B, C, K] times w [B, N, K]: products of a batch."""
    return torch.matmul(x, w.transpose(1, 2).contiguous())


# ------------------------------------------------------------------ inputs ----

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _weights(g, *shape):
    """MXFP4 codes and scales of normal weights whose rows and blocks differ in size."""
    lead, K = shape[:-1], shape[-1]
    w = torch.randn(*lead, K, generator=g, device="cuda") * (1.0 / math.sqrt(K))
    w = w.reshape(*lead, K // 32, 32)
    w = w * torch.exp2(torch.rand(*lead, K // 32, 1, generator=g, device="cuda") * 3 - 1.5)
    return _quantize(w.reshape(*lead, K))


def _acts(g, R, K, dtype):
    """Activations: normal, with some channels that stand out."""
    x = torch.randn(R, K, generator=g, device="cuda")
    loud = torch.rand(K, generator=g, device="cuda") < 0.01
    return (x * torch.where(loud, 8.0, 1.0)).to(dtype)


def prepare(case, seed):
    c, g = case, _gen(seed)
    op = c["op"]
    s = {"case": c, "op": op}
    if op == "quantize":
        s["x"] = _acts(g, c["R"], c["K"], DTYPES[c["type"]])
    elif op == "linear":
        s["x"] = _acts(g, c["M"], c["K"], DTYPES[c["type"]])
        s["w"], s["s"] = _weights(g, c["N"], c["K"])
        s["residual"] = _acts(g, c["M"], c["N"], DTYPES[c["type"]]) if c["residual"] else None
        s["dtype"] = DTYPES[c["out"]]
    elif op == "matmul":
        s["a"], s["sa"] = _quantize(_acts(g, c["M"], c["K"], torch.bfloat16))
        s["w"], s["s"] = _weights(g, c["N"], c["K"])
        s["dtype"] = DTYPES[c["out"]]
    elif op == "route":
        s["logits"] = (2.0 * torch.randn(c["T"], c["E"], generator=g, device="cuda")).to(DTYPES[c["type"]])
        s["k"], s["scoring"] = c["k"], c["scoring"]
    elif op == "experts":
        T, E, k, H, I = c["T"], c["E"], c["k"], c["H"], c["I"]
        s["x"] = _acts(g, T, H, DTYPES[c["type"]])
        lean = torch.randn(E, generator=g, device="cuda") * 0.7    # some experts are chosen more often
        lo = torch.randn(T, E, generator=g, device="cuda") + lean
        top = torch.sort(lo, dim=-1, descending=True, stable=True)
        s["ids"] = top.indices[:, :k].to(torch.int32).contiguous()
        s["weights"] = torch.softmax(top.values[:, :k], -1).contiguous()
        s["wg"], s["sg"] = _weights(g, E, I, H)
        s["wu"], s["su"] = _weights(g, E, I, H)
        s["wd"], s["sd"] = _weights(g, E, H, I)
        s["residual"] = _acts(g, T, H, DTYPES[c["type"]]) if c["residual"] else None
    else:
        P, E = c["P"], c["E"]
        s["x"] = _acts(g, P, c["K"], DTYPES[c["type"]])
        s["w"], s["s"] = _weights(g, E, c["N"], c["K"])
        share = torch.rand(E, generator=g, device="cuda") + 0.2
        if c["skew"]:        # a few experts take most rows, about a quarter of them none
            share = torch.exp(1.5 * torch.randn(E, generator=g, device="cuda"))
            share[torch.rand(E, generator=g, device="cuda") < 0.25] = 0.0
            share[E // 2] += 0.1
        at = torch.cumsum(share, 0) / share.sum() * P
        s["offsets"] = torch.cat([torch.zeros(1, device="cuda"), at[:-1].round(),
                                  torch.full((1,), float(P), device="cuda")]).to(torch.int32)
        s["dtype"] = DTYPES[c["out"]]
    return s


# --------------------------------------------------------------------- run ----

def run(s):
    op = s["op"]
    if own:
        swq = calls()
        if op == "quantize":
            return swq.mx4_dequantize(*swq.mx4_quantize(s["x"]), s["x"].dtype)
        if op == "linear":
            return swq.mx4_linear(s["x"], s["w"], s["s"], residual=s["residual"], out_mode=OUT_MODE[s["dtype"]])
        if op == "matmul":
            return swq.mx4_matmul(s["a"], s["sa"], s["w"], s["s"], out_mode=OUT_MODE[s["dtype"]])
        if op == "route":
            return swq.route(s["logits"], s["k"], SCORING[s["scoring"]])
        if op == "experts":
            return swq.moe_mlp(s["x"], s["ids"], s["weights"], s["wg"], s["sg"], s["wu"], s["su"], s["wd"], s["sd"],
                               residual=s["residual"])
        return swq.mx4_grouped_linear(s["x"], s["offsets"], s["w"], s["s"], out_mode=OUT_MODE[s["dtype"]])

    if op == "quantize":
        return _values(*_quantize(s["x"])).to(s["x"].dtype)
    if op == "linear":
        y = torch.matmul(s["x"].float(), _values(s["w"], s["s"]).t())
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return y.to(s["dtype"])
    if op == "matmul":
        return torch.matmul(_values(s["a"], s["sa"]), _values(s["w"], s["s"]).t()).to(s["dtype"])
    if op == "route":
        top = torch.sort(s["logits"].float(), dim=-1, descending=True, stable=True)
        ids, v = top.indices[:, :s["k"]], top.values[:, :s["k"]]
        if s["scoring"] == "softmax":
            p = torch.exp(v - top.values[:, :1]) / torch.exp(top.values - top.values[:, :1]).sum(-1, keepdim=True)
        elif s["scoring"] == "softmax_chosen":
            p = torch.exp(v - v[:, :1])
            p = p / p.sum(-1, keepdim=True)
        else:
            p = 1.0 / (1.0 + torch.exp(-v))
            if s["scoring"] == "sigmoid_chosen":
                p = p / p.sum(-1, keepdim=True)
        return ids.to(torch.int32), p
    if op == "experts":
        T, k = s["ids"].shape
        x = s["x"].float()
        rows, valid, pick = _table(s["ids"].reshape(-1).long(), s["wg"].shape[0], T * k <= 32)
        xr = x[rows // k]
        h = _silu(_times(xr, _values(s["wg"][pick], s["sg"][pick]))) * _times(xr, _values(s["wu"][pick], s["su"][pick]))
        y = _scatter(_times(h, _values(s["wd"][pick], s["sd"][pick])), rows, valid, T * k)
        y = (y.reshape(T, k, -1) * s["weights"][..., None]).sum(1)
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return y.to(s["x"].dtype)
    P, E = s["x"].shape[0], s["w"].shape[0]
    expert = (torch.arange(P, device="cuda")[:, None] >= s["offsets"][None, 1:]).sum(1)
    rows, valid, pick = _table(expert, E, P <= 32)
    y = _times(s["x"].float()[rows], _values(s["w"][pick], s["s"][pick]))
    return _scatter(y, rows, valid, P).to(s["dtype"])


# ------------------------------------------------------------------- exact ----

def _wide(codes, scales):
    """Values in 64 bits from the bits of the format: sign, two exponent bits, one fraction bit."""
    n = codes.shape[-1]
    q = torch.stack([torch.bitwise_and(torch.bitwise_right_shift(codes.long(), 4 * j), 15) for j in range(8)], -1)
    q = q.reshape(*codes.shape[:-1], 8 * n)
    ex, fr = torch.div(q % 8, 2, rounding_mode="floor"), (q % 2).double()
    mag = torch.where(ex == 0, 0.5 * fr, (1.0 + 0.5 * fr) * torch.pow(2.0, (ex - 1).double()))
    v = torch.where(q >= 8, -mag, mag)
    p = torch.pow(torch.tensor(2.0, dtype=torch.float64, device=v.device), scales.double() - 127.0)
    return v * p.repeat_interleave(32, -1)


def _nearest(x):
    """x rounded to the nearest value of the format, block by block, in 64 bits."""
    b = x.double().reshape(-1, 32)
    top = b.abs().amax(-1, keepdim=True)
    e = torch.floor(torch.log2(torch.where(top > 0, top, torch.ones_like(top))))
    unit = torch.pow(2.0, torch.clamp(e - 2.0, min=-127.0))
    a = b / unit
    step = torch.pow(2.0, torch.clamp(torch.floor(torch.log2(a.abs().clamp(min=1.0))), min=0.0) - 1.0)
    r = (torch.round(a / step) * step).clamp(-6.0, 6.0)
    return (r * unit).reshape(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "quantize":
        return _nearest(s["x"])
    if op == "linear":
        y = s["x"].double() @ _wide(s["w"], s["s"]).t()
        return y if s["residual"] is None else y + s["residual"].double()
    if op == "matmul":
        return _wide(s["a"], s["sa"]) @ _wide(s["w"], s["s"]).t()
    if op == "route":
        lo, k = s["logits"].double(), s["k"]
        n = torch.arange(lo.shape[1], device=lo.device).double()
        left = lo.clone()
        ids = []
        for _ in range(k):
            best = left.amax(-1, keepdim=True)
            at = torch.where(left == best, n, float("inf")).amin(-1, keepdim=True).long()
            ids.append(at)
            left.scatter_(1, at, float("-inf"))
        ids = torch.cat(ids, -1)
        v = lo.gather(1, ids)
        if s["scoring"].startswith("softmax"):
            over = lo if s["scoring"] == "softmax" else v
            return None, torch.exp(v - torch.logsumexp(over, -1, keepdim=True))
        p = torch.sigmoid(v)
        return None, p if s["scoring"] == "sigmoid" else p / p.sum(-1, keepdim=True)
    if op == "experts":
        ids, x = s["ids"].long(), s["x"].double()
        y = torch.zeros_like(x) if s["residual"] is None else s["residual"].double()
        for e in torch.unique(ids).tolist():
            t, j = torch.nonzero(ids == e, as_tuple=True)
            g = x[t] @ _wide(s["wg"][e], s["sg"][e]).t()
            h = g * torch.sigmoid(g) * (x[t] @ _wide(s["wu"][e], s["su"][e]).t())
            y.index_add_(0, t, (h @ _wide(s["wd"][e], s["sd"][e]).t()) * s["weights"][t, j].double()[:, None])
        return y
    at = s["offsets"].tolist()
    return torch.cat([s["x"][a:b].double() @ _wide(s["w"][e], s["s"][e]).t()
                      for e, (a, b) in enumerate(zip(at[:-1], at[1:])) if b > a])
