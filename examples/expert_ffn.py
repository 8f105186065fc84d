"""A feed-forward layer of experts on the library's operators: RMS norm of the residual
stream, router product, each token's choice of experts, the rows sorted by expert,
gated products of each expert's rows in 8-bit floating point, and the weighted sum
back in token order.  Nothing of it waits for the host, so a decoded step is one CUDA
graph; the way back gives the gradients of the rows and of the router's logits.

    python examples/expert_ffn.py --width 2048 --hidden 1024 --experts 64 --top 8 --tokens 16
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from dit_convrot_linear_gb300 import tq  # noqa: E402


class Experts:
    def __init__(self, width, hidden, experts, top, seed=0):
        import torch
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.hidden, self.experts, self.top = hidden, experts, top
        self.gamma = 1.0 + 0.1 * torch.randn(width, generator=g, device="cuda")
        self.weights, self.plain = {}, {}    # plain: bf16, for the comparison below
        for name, n, k in (("router", experts, width), ("up", 2 * hidden, width), ("down", width, hidden)):
            shape = (n, k) if name == "router" else (experts, n, k)
            self.plain[name] = (torch.randn(*shape, generator=g, device="cuda") * k ** -0.5).bfloat16()
            self.weights[name] = tq.quantize_weights_f8(self.plain[name])
        self.workspace = tq.f8_workspace()

    def route(self, x):
        """(logits, ids, weights) of bf16 rows x."""
        logits = tq.linear_f8(*tq.quant_act_f8(x), *self.weights["router"], self.workspace, out="f32")
        return (logits, *tq.expert_topk(logits, self.top))

    def __call__(self, x, residual):
        """(output, residual) of bf16 [tokens, width]; what the way back needs stays in
        ``saved``."""
        import torch
        total = torch.empty_like(x)
        x = tq.rmsnorm(x, self.gamma, R=residual, H=total)
        logits, ids, weights = self.route(x)
        offsets, token, place = tq.expert_sort(ids, self.experts)
        q, s = tq.quant_act_f8(x, rows=token)
        gu = tq.linear_f8_experts(q, s, offsets, *self.weights["up"], self.workspace)
        q, s = tq.swiglu_quant_act_f8(gu[:, :self.hidden], gu[:, self.hidden:])
        y = tq.linear_f8_experts(q, s, offsets, *self.weights["down"], self.workspace)
        self.saved = x, logits, ids, weights, place, y
        return tq.expert_combine(y, place, weights), total

    def backward(self, dO):
        """(gradient of the experts' rows, of the router's logits) from the output's."""
        _, logits, ids, weights, place, y = self.saved
        dy, dw = tq.expert_combine_grad(dO, y, place, weights)
        return dy, tq.expert_topk_grad(logits, ids, dw)

    def exact(self, x, ids, weights):
        """The experts' sum in fp32, for these choices."""
        import torch
        out = torch.zeros(x.shape, device="cuda")
        up, down = self.plain["up"], self.plain["down"]
        for e in range(self.experts):
            t, j = (ids == e).nonzero(as_tuple=True)
            if t.numel():
                v = x[t].float() @ up[e].float().t()
                g, u = v[:, :self.hidden], v[:, self.hidden:]
                out.index_add_(0, t, weights[t, j, None] * ((g * torch.sigmoid(g) * u) @ down[e].float().t()))
        return out


def run(width=512, hidden=256, experts=16, top=4, tokens=16, steps=4, seed=0):
    """Relative error of the output against fp32, the largest difference between a
    captured step and the same step by itself, and a step's time in us."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    layer = Experts(width, hidden, experts, top, seed)
    xs = torch.randn(steps, tokens, width, generator=g, device="cuda").bfloat16()
    rs = torch.randn(steps, tokens, width, generator=g, device="cuda").bfloat16()
    x, r = xs[0].clone(), rs[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())       # the weights and rows are made there
    with torch.cuda.stream(side):
        layer(x, r)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _ = layer(x, r)
    saved = layer.saved
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    num = den = differ = 0.0
    times = []
    for i in range(steps):
        x.copy_(xs[i])
        r.copy_(rs[i])
        begin.record()
        graph.replay()
        end.record()
        end.synchronize()
        times.append(1e3 * begin.elapsed_time(end))
        want = layer.exact(saved[0], saved[2], saved[3])
        num += float((out.float() - want).pow(2).sum())
        den += float(want.pow(2).sum())
        differ = max(differ, float((layer(x, r)[0].float() - out.float()).abs().max()))
    if tq.device_status() != 0:
        raise RuntimeError("the device reported an error")
    return (num / den) ** 0.5, differ, sorted(times)[len(times) // 2]


def main():
    a = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    for name, v in (("width", 2048), ("hidden", 1024), ("experts", 64), ("top", 8), ("tokens", 16), ("steps", 16)):
        a.add_argument("--" + name, type=int, default=v)
    a = a.parse_args()
    err, differ, us = run(a.width, a.hidden, a.experts, a.top, a.tokens, a.steps)
    print(f"{a.tokens} tokens, {a.top} of {a.experts} experts each: relative error against fp32 {err:.4f}")
    print(f"graph against single launches: {differ}")
    print(f"a step of the layer: {us:.1f} us")


if __name__ == "__main__":
    main()
