"""Cases of the operators with 16-bit weights and of training: the dense linear
with bias, activation and residual and its gradients, 8-bit activation
checkpoints, the SwiGLU that leaves such checkpoints behind with its gradient,
the router's balance loss and gradient.  What each computes in elementary torch
operations, and the calls a user makes.

Checkpoint format: int8 codes q, one e8m0 byte b per 32 neighbours of a row (the
last block of a row may be shorter), value q 2^(b - 133); steps from 2^-126 on.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
OUT_MODE = {"bf16": 0, "f32": 1, "f16": 2}                                      # the library's SWQ_LINEAR_*
ACT = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}              # its SWQ_ACT_*
SCORING = {"softmax": 0, "softmax_chosen": 1, "sigmoid": 2, "sigmoid_chosen": 3}    # its SWQ_ROUTE_*
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
MX8_BYTES = 1.0 + 1.0 / 32.0     # of one element: its code and its share of a scale


def calls():
    import quantized_swiglu_forward_amd as swq
    return swq


# ------------------------------------------------------------------- cases ----

def listed():
    return [
        # decode: one token through an unquantised projection
        {"name": "linear-1x2048x5632", "op": "linear", "M": 1, "K": 2048, "N": 5632, "type": "bf16", "out": "bf16",
         "act": "silu", "bias": True, "residual": False},
        # a small batch, sizes that are no multiple of anything, float32 sums returned
        {"name": "linear-37x1003x2049", "op": "linear", "M": 37, "K": 1003, "N": 2049, "type": "f16", "out": "f32",
         "act": "none", "bias": True, "residual": True},
        # prefill: a wide expansion with its activation
        {"name": "linear-2048x4096x14336", "op": "linear", "M": 2048, "K": 4096, "N": 14336, "type": "bf16",
         "out": "bf16", "act": "gelu", "bias": True, "residual": True},
        # one small layer's training step, ragged, what the backward pass needs kept in 16 bits
        {"name": "train-77x517x1001", "op": "train", "M": 77, "K": 517, "N": 1001, "type": "f16", "act": "gelu",
         "keep": "same", "residual": False},
        # a middle-sized layer's training step, 8-bit checkpoints
        {"name": "train-2048x2048x5632", "op": "train", "M": 2048, "K": 2048, "N": 5632, "type": "bf16",
         "act": "gelu_tanh", "keep": "mx8", "residual": False},
        # the large expansion's training step, 8-bit checkpoints
        {"name": "train-2048x4096x14336", "op": "train", "M": 2048, "K": 4096, "N": 14336, "type": "bf16",
         "act": "silu", "keep": "mx8", "residual": True},
        # a small batch's activations written as checkpoints and read back
        {"name": "checkpoint-48x2048", "op": "checkpoint", "R": 48, "K": 2048, "type": "bf16"},
        # a long prefill's hidden tensor, the same
        {"name": "checkpoint-8192x10240", "op": "checkpoint", "R": 8192, "K": 10240, "type": "bf16"},
        # the SwiGLU between a small layer's projections, forward with checkpoints and backward from them
        {"name": "swiglu-6x768", "op": "swiglu", "R": 6, "K": 768, "type": "bf16"},
        # the same of a large layer
        {"name": "swiglu-2048x14336", "op": "swiglu", "R": 2048, "K": 14336, "type": "bf16"},
        # a small batch's router: loss, counts and the logits' gradient
        {"name": "router-65x64-top4", "op": "router", "T": 65, "E": 64, "k": 4, "type": "f32",
         "scoring": "sigmoid_chosen"},
        # a long prefill's router, many experts
        {"name": "router-8192x256-top8", "op": "router", "T": 8192, "E": 256, "k": 8, "type": "bf16",
         "scoring": "softmax"},
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
        op = rng.choice(["linear", "train", "checkpoint", "swiglu", "router"])
        t = rng.choice(["bf16", "bf16", "f16"])
        if op == "linear":
            c = {"M": _log(rng, 1, 8192), "K": _log(rng, 16, 14336), "N": _log(rng, 4, 14336), "type": t,
                 "out": rng.choice([t, t, "f32"]), "act": rng.choice(list(ACT)), "bias": rng.random() < 0.7,
                 "residual": rng.random() < 0.5}
        elif op == "train":
            c = {"M": _log(rng, 1, 8192), "K": _log(rng, 16, 8192), "N": _log(rng, 4, 14336), "type": t,
                 "act": rng.choice(list(ACT)), "keep": rng.choice(["mx8", "same"]), "residual": rng.random() < 0.5}
        elif op == "checkpoint":
            c = {"R": _log(rng, 1, 16384), "K": _log(rng, 16, 14336), "type": rng.choice(["bf16", "f16", "f32"])}
        elif op == "swiglu":
            c = {"R": _log(rng, 1, 8192), "K": _log(rng, 32, 14336), "type": t}
        else:
            E = _log(rng, 4, 512)
            c = {"T": _log(rng, 1, 8192), "E": E, "k": rng.randint(1, min(10, E)),
                 "type": rng.choice(["bf16", "f16", "f32"]), "scoring": rng.choice(list(SCORING))}
        c = {"op": op, **c}
        w = work(c)
        if w["bytes"] <= most[op][0] and w["flops"] <= most[op][1]:
            return c


def work(c):
    """Each input of a call once, each output once (what the forward call leaves for the backward one among them)."""
    op = c["op"]
    if op == "checkpoint":      # in, codes and scales out; codes and scales in, values out
        return {"bytes": c["R"] * c["K"] * 2 * (SIZE[c["type"]] + MX8_BYTES), "flops": 0}
    if op == "swiglu":          # gate, up in, hidden and checkpoints out; dhidden and checkpoints in, three out
        return {"bytes": c["R"] * c["K"] * (3 * 2 + 2 * MX8_BYTES + 2 + 2 * MX8_BYTES + 3 * 2), "flops": 0}
    if op == "router":
        T, E, k = c["T"], c["E"], c["k"]
        return {"bytes": 3 * T * E * SIZE[c["type"]] + T * k * (4 + 4 + 4) + E * 12, "flops": 0}
    M, K, N = c["M"], c["K"], c["N"]
    if op == "linear":
        return {"bytes": 2 * (M * K + N * K) + M * N * (SIZE[c["out"]] + (2 if c["residual"] else 0))
                + (2 * N if c["bias"] else 0), "flops": 2 * M * N * K}
    keep = MX8_BYTES if c["keep"] == "mx8" else 2
    z = 0 if c["act"] == "none" else 2 * M * N * keep
    x = M * K * (2 * keep + 2 if c["keep"] == "mx8" else 2)
    forward = M * K * 2 + N * K * 2 + N * 2 + M * N * (4 if c["residual"] else 2)
    return {"bytes": forward + z + x + M * N * 2 + N * K * 4 + M * K * 2 + N * 2, "flops": 6 * M * N * K}


# --------------------------------------------------------- elementary parts ----

def _power(e):
    """2^e of whole numbers in [-126, 127], exact (a power function may be off by a bit, which moves ties)."""
    return ((e + 127) << 23).view(torch.float32)


def _checkpoint(x):
    """The values that x's 8-bit checkpoint stands for, in float32."""
    K = x.shape[-1]
    pad = -K % 32
    b = x.float()
    if pad:
        b = torch.cat([b, b.new_zeros(*b.shape[:-1], pad)], -1)
    b = b.reshape(*x.shape[:-1], -1, 32)
    amax = b.abs().amax(-1, keepdim=True)
    e = (torch.frexp(amax).exponent - 7).clamp(min=-126)            # amax in [64, 128) steps of 2^e
    e = e + (torch.round(amax * _power(-e)) > 127).int()
    return (torch.round(b * _power(-e)) * _power(e)).reshape(*x.shape[:-1], K + pad)[..., :K]


def _sigma(t):
    return 1.0 / (1.0 + torch.exp(-t))


_C0, _C1 = math.sqrt(2.0 / math.pi), 0.044715


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "silu":
        return z * _sigma(z)
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(_C0 * (z + _C1 * z * z * z)))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        s = _sigma(z)
        return s * (1.0 + z * (1.0 - s))
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * math.sqrt(0.5 / math.pi)
    if act == "gelu_tanh":
        t = torch.tanh(_C0 * (z + _C1 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * _C0 * (1.0 + 3.0 * _C1 * z * z)
    return torch.ones_like(z)


def _router(logits, ids, dw, dloss, scoring):
    """(loss, counts, dlogits), every token with k experts."""
    T, E = logits.shape
    k = ids.shape[1]
    lo = logits.float()
    ix = ids.long()
    hot = (ix[:, :, None] == torch.arange(E, device=ix.device)).float()       # [T, k, E]
    counts = hot.sum((0, 1)).to(torch.int32)
    soft = torch.exp(lo - lo.amax(-1, keepdim=True))
    soft = soft / soft.sum(-1, keepdim=True)
    s = _sigma(lo)
    p = soft if scoring.startswith("softmax") else s / s.sum(-1, keepdim=True)
    f = counts.float() / (T * k)
    loss = E * (f * p.mean(0)).sum()
    v = dloss * E * f / T
    d = p * (v - (v * p).sum(-1, keepdim=True))
    if not scoring.startswith("softmax"):
        d = d * (1.0 - s)
    if scoring == "softmax":
        each = (hot * dw[:, :, None]).sum(1)
        d = d + soft * (each - (each * soft).sum(-1, keepdim=True))
    else:
        of = torch.exp(lo.gather(1, ix) - lo.gather(1, ix).amax(-1, keepdim=True)) if scoring == "softmax_chosen" \
            else s.gather(1, ix)
        if scoring == "sigmoid":
            g = dw * of * (1.0 - of)
        else:
            w = of / of.sum(-1, keepdim=True)
            g = w * (dw - (w * dw).sum(-1, keepdim=True))
            if scoring == "sigmoid_chosen":
                g = g * (1.0 - of)
        d = d + (hot * g[:, :, None]).sum(1)
    return loss, counts, d.to(logits.dtype)


# ------------------------------------------------------------------ inputs ----

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _acts(g, R, K, dtype):
    """Activations: normal, with some channels that stand out."""
    x = torch.randn(R, K, generator=g, device="cuda")
    loud = torch.rand(K, generator=g, device="cuda") < 0.01
    return (x * torch.where(loud, 8.0, 1.0)).to(dtype)


def prepare(case, seed):
    c, g = case, _gen(seed)
    op = c["op"]
    s = {"case": c, "op": op}
    t = DTYPES[c["type"]]
    if op == "checkpoint":
        s["x"] = _acts(g, c["R"], c["K"], t)
    elif op == "swiglu":
        s["gate"], s["up"] = _acts(g, c["R"], c["K"], t), _acts(g, c["R"], c["K"], t)
        s["dhidden"] = torch.randn(c["R"], c["K"], generator=g, device="cuda").to(t)
    elif op == "router":
        lean = 0.5 * torch.randn(c["E"], generator=g, device="cuda")         # some experts are chosen more often
        s["logits"] = (1.5 * torch.randn(c["T"], c["E"], generator=g, device="cuda") + lean).to(t)
        order = torch.sort(s["logits"].float(), dim=-1, descending=True, stable=True).indices
        s["ids"] = order[:, :c["k"]].to(torch.int32).contiguous()
        s["dweights"] = torch.randn(c["T"], c["k"], generator=g, device="cuda")
        s["dloss"] = torch.full((), 0.01 * c["T"], device="cuda")       # the loss's factor beside a sum over tokens
    else:
        M, K, N = c["M"], c["K"], c["N"]
        s["x"] = _acts(g, M, K, t)
        s["w"] = (torch.randn(N, K, generator=g, device="cuda") / math.sqrt(K)).to(t)
        s["bias"] = (0.2 * torch.randn(N, generator=g, device="cuda")).to(t) if c.get("bias", True) else None
        s["residual"] = _acts(g, M, N, t) if c["residual"] else None
        if op == "train":
            s["dout"] = torch.randn(M, N, generator=g, device="cuda").to(t)
    return s


# --------------------------------------------------------------------- run ----

def run(s):
    op, c = s["op"], s["case"]
    if own:
        swq = calls()
        if op == "checkpoint":
            return swq.mx8_dequantize(*swq.mx8_quantize(s["x"]), s["x"].dtype)
        if op == "swiglu":
            hidden, gate, up = swq.swiglu(s["gate"], s["up"], keep=True)
            dgate, dup, again = swq.swiglu_backward(s["dhidden"], gate, up, hidden=True)
            return hidden, dgate, dup, again
        if op == "router":
            scoring = SCORING[c["scoring"]]
            loss, counts, slopes = swq.balance_loss(s["logits"], s["ids"], scoring)
            return loss, counts, swq.route_backward(s["logits"], s["ids"], s["dweights"], scoring, slopes=slopes,
                                                    dloss=s["dloss"])
        act = ACT[c["act"]]
        if op == "linear":
            return swq.dense_linear(s["x"], s["w"], s["bias"], act=act, residual=s["residual"],
                                    out_mode=OUT_MODE[c["out"]])
        mx8 = c["keep"] == "mx8"
        if c["act"] == "none":
            out, z = swq.dense_linear(s["x"], s["w"], s["bias"], residual=s["residual"]), None
        else:
            out, z = swq.dense_linear(s["x"], s["w"], s["bias"], act=act, residual=s["residual"],
                                      keep="mx8" if mx8 else "same")
        x = swq.mx8_quantize(s["x"]) if mx8 else s["x"]
        return (out, *swq.dense_linear_backward(s["dout"], x, s["w"], z, act=act))

    if op == "checkpoint":
        return _checkpoint(s["x"]).to(s["x"].dtype)
    if op == "swiglu":
        t = s["gate"].dtype
        g, u = s["gate"].float(), s["up"].float()
        hidden = (g * _sigma(g) * u).to(t)
        g, u, d = _checkpoint(s["gate"]), _checkpoint(s["up"]), s["dhidden"].float()
        q = _sigma(g)
        return hidden, (d * u * q * (1.0 + g * (1.0 - q))).to(t), (d * g * q).to(t), (g * q * u).to(t)
    if op == "router":
        return _router(s["logits"], s["ids"], s["dweights"], s["dloss"], c["scoring"])
    x, w = s["x"].float(), s["w"].float()
    z = torch.matmul(x, w.t())
    if s["bias"] is not None:
        z = z + s["bias"].float()
    out = _act(z, c["act"])
    if s["residual"] is not None:
        out = out + s["residual"].float()
    if op == "linear":
        return out.to(DTYPES[c["out"]])
    t = s["x"].dtype
    if c["keep"] == "mx8":
        z, x = _checkpoint(z), _checkpoint(x)
    else:
        z = z.to(t).float()
    dz = s["dout"].float() * _act_slope(z, c["act"])
    return out.to(t), torch.matmul(dz, w).to(t), torch.matmul(dz.t(), x).to(t), dz.sum(0).to(t)


# ------------------------------------------------------------------- exact ----

def _nearest(x):
    """x on the checkpoint's grid, row by row, in 64 bits: the finest power-of-two step at which 127 steps hold a block."""
    v = x.double()
    at = torch.div(torch.arange(v.shape[-1], device=v.device), 32, rounding_mode="floor")
    blocks = int(at[-1]) + 1
    top = torch.zeros(v.shape[0], blocks, dtype=torch.float64, device=v.device)
    top = top.scatter_reduce(1, at.expand(v.shape[0], -1), v.abs(), "amax")
    bits = top.clamp(min=2.0 ** -120).view(torch.int64) & (0x7FF << 52)     # the largest element's power of two
    step = bits.view(torch.float64) / 64.0
    step = torch.where(torch.round(top / step) >= 128.0, 2.0 * step, step)[:, at]
    return torch.round(v / step) * step


def _wide_act(z, act):
    """(act(z), its derivative) in 64 bits."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return z.clamp(min=0.0), torch.heaviside(z, torch.zeros_like(z))
    if act == "silu":
        s = torch.sigmoid(z)
        return z * s, s + z * s * torch.sigmoid(-z)
    if act == "gelu":
        phi = 0.5 * torch.special.erfc(-z / math.sqrt(2.0))
        return z * phi, phi + z * torch.exp(-z * z / 2.0) / math.sqrt(2.0 * math.pi)
    u = math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)
    s = torch.sigmoid(2.0 * u)                                    # (1 + tanh u) / 2
    return z * s, s + 2.0 * z * s * (1.0 - s) * math.sqrt(2.0 / math.pi) * (1.0 + 3.0 * 0.044715 * z ** 2)


def exact(case, seed):
    s = prepare(case, seed)
    op, c = s["op"], case
    if op == "checkpoint":
        return _nearest(s["x"])
    if op == "swiglu":
        a, _ = _wide_act(s["gate"].double(), "silu")
        b, slope = _wide_act(_nearest(s["gate"]), "silu")
        u, d = _nearest(s["up"]), s["dhidden"].double()
        return a * s["up"].double(), d * u * slope, d * b, b * u
    if op == "router":
        # the loss as a function of the logits, and its derivative by the graph
        lo = s["logits"].double().requires_grad_(True)
        ix = s["ids"].long()
        T, E, k = c["T"], c["E"], c["k"]
        f = torch.bincount(ix.reshape(-1), minlength=E).double() / (T * k)
        soft = torch.exp(lo - torch.logsumexp(lo, -1, keepdim=True))
        sig = torch.sigmoid(lo)
        p = soft if c["scoring"].startswith("softmax") else sig / sig.sum(-1, keepdim=True)
        loss = E * (f * p.sum(0) / T).sum()
        if c["scoring"] == "softmax":
            w = soft.gather(1, ix)
        elif c["scoring"] == "softmax_chosen":
            v = lo.gather(1, ix)
            w = torch.exp(v - torch.logsumexp(v, -1, keepdim=True))
        else:
            w = sig.gather(1, ix)
            if c["scoring"] == "sigmoid_chosen":
                w = w / w.sum(-1, keepdim=True)
        (s["dloss"].double() * loss + (w * s["dweights"].double()).sum()).backward()
        return loss.detach(), None, lo.grad
    z = s["x"].double() @ s["w"].double().t()
    if s["bias"] is not None:
        z = z + s["bias"].double()
    out = _wide_act(z, c["act"])[0]
    if s["residual"] is not None:
        out = out + s["residual"].double()
    if op == "linear":
        return out
    x = s["x"]
    if c["keep"] == "mx8":
        z, x = _nearest(z), _nearest(x)
    else:
        z, x = z.to(x.dtype).double(), x.double()
    dz = s["dout"].double() * _wide_act(z, c["act"])[1]
    return out, dz @ s["w"].double(), dz.t() @ x, dz.sum(0)
