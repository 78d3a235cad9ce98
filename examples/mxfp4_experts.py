"""A layer of MXFP4 experts, as a model would hold and call it.

    python examples/mxfp4_experts.py [--tokens 512] [--hidden 2048] [--intermediate 1024]
                                     [--experts 64] [--chosen 8]

The layer quantizes its experts' weights once, and each call routes its tokens
and runs their experts' MLPs with the residual.  It prints how far the quantized layer
is from the same layer in float32, and the time of a prefill call and of a decode
step (one token, replayed from a HIP graph as a serving loop would).
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import quantized_swiglu_forward_amd as swq  # noqa: E402


class Experts:
    """Router weights [E, H] (bf16) and the experts' gate, up and down weights as MXFP4."""

    def __init__(self, router, gate, up, down, chosen):
        self.router, self.chosen = router, chosen
        self.gate, self.up, self.down = (swq.mx4_quantize(w) for w in (gate, up, down))

    def __call__(self, x, out=None):
        logits = torch.matmul(x, self.router.t())
        ids, weights = swq.route(logits, self.chosen, swq.SWQ_ROUTE_SOFTMAX_CHOSEN)
        return swq.moe_mlp(x, ids, weights, *self.gate, *self.up, *self.down, residual=x, out=out)


def float_layer(x, router, gate, up, down, chosen):
    logits = torch.matmul(x, router.t()).float()
    top = torch.topk(logits, chosen)
    weights = torch.softmax(top.values, -1)
    y = x.float().clone()
    for e in range(gate.shape[0]):
        t, j = torch.nonzero(top.indices == e, as_tuple=True)
        if t.numel():
            h = torch.nn.functional.silu(x[t].float() @ gate[e].t()) * (x[t].float() @ up[e].t())
            y.index_add_(0, t, (h @ down[e].t()) * weights[t, j][:, None])
    return y


def microseconds(call, n=50):
    for _ in range(5):
        call()
    torch.cuda.synchronize()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(n):
        call()
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b) * 1e3 / n


def main():
    ap = argparse.ArgumentParser(description=__doc__)
    for name, value in (("tokens", 512), ("hidden", 2048), ("intermediate", 1024), ("experts", 64), ("chosen", 8)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    g = torch.Generator(device="cuda").manual_seed(0)

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * scale

    E, H, I = a.experts, a.hidden, a.intermediate
    router = normal(E, H, scale=H ** -0.5).bfloat16()
    gate, up, down = normal(E, I, H, scale=H ** -0.5), normal(E, I, H, scale=H ** -0.5), normal(E, H, I, scale=I ** -0.5)
    layer = Experts(router, gate, up, down, a.chosen)

    x = normal(a.tokens, H).bfloat16()
    y, want = layer(x).float(), float_layer(x, router, gate, up, down, a.chosen)
    print(f"relative difference from float32 weights: {float((y - want).norm() / (want - x.float()).norm()):.3f}")
    print(f"{a.tokens} tokens: {microseconds(lambda: layer(x)):.1f} us")

    one = x[:1].contiguous()
    out = torch.empty_like(one)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        layer(one, out=out)              # the workspace has its size before the capture
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        layer(one, out=out)
    print(f"one token, from a graph: {microseconds(graph.replay):.1f} us")


if __name__ == "__main__":
    main()
