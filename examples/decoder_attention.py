"""One attention layer of a decoder on the library's operators: RMS norm of the
residual stream, query/key/value product, rotary positions, 4-bit cache,
attention over it, output product.  Prompts go through as one ragged batch (A8
products on tiled operands), decoded tokens a token a sequence (A16 products), as
one CUDA graph whose lengths and positions live on the device.

    python examples/decoder_attention.py --width 4096 --heads 32 --heads-kv 8 --dim 128 --batch 64 --prompt 1024
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from dit_convrot_linear_gb300 import tq  # noqa: E402

DECODE_ROWS = 64                             # the A16 products take as many


class Attention:
    def __init__(self, width, heads, heads_kv, dim, theta=10000.0, seed=0):
        import torch
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.width, self.heads, self.heads_kv, self.dim = width, heads, heads_kv, dim
        self.scale = dim ** -0.5
        self.gamma = 1.0 + 0.1 * torch.randn(width, generator=g, device="cuda")
        self.weights = {}                    # fp32, for the comparison below
        for name, n, k in (("qkv", (heads + 2 * heads_kv) * dim, width), ("out", width, heads * dim)):
            W = torch.randn(n, k, generator=g, device="cuda") * k ** -0.5
            codes, scales = tq.quantize_weights(W.bfloat16(), 8)
            self.weights[name] = (W.bfloat16().float(), codes, scales, tq.tile_weights(codes, n, k, 8))
        inv = theta ** (-torch.arange(0, dim, 2, device="cuda", dtype=torch.float32) / dim)
        self.rope = tq.RopeSpec(inv)
        self.inv_freq = inv
        self.workspace = tq.kv4_workspace()

    def product(self, name, X=None, At=None, sx=None, rows=None):
        """bf16 rows of a weight's product: of X, or of a tiled operand."""
        _, codes, scales, tiles = self.weights[name]
        n, k = self.weights[name][0].shape
        if At is None and X.shape[0] <= DECODE_ROWS:
            return tq.linear(X, codes, scales, n, 8, "W8A16", out="bf16")
        if At is None:
            rows = X.shape[0]
            At, sx = tq.rotate_quant_act_tiled(X)
        return tq.linear_tt(At, sx, rows, k, tiles, scales, n, 8, out="bf16")

    def __call__(self, x, residual, batch, pos):
        """(output, residual): x and residual bf16 [tokens, width], pos int32 [1,
        tokens]; the batch's cache gains the tokens' keys and values."""
        import torch
        M, H, D = x.shape[0], self.heads, self.dim
        total = torch.empty_like(x)
        if M <= DECODE_ROWS:
            qkv = self.product("qkv", tq.rmsnorm(x, self.gamma, R=residual, H=total))
        else:
            At, sx = tq.rmsnorm_quant_act_tiled(x, self.gamma, R=residual, H=total)
            qkv = self.product("qkv", At=At, sx=sx, rows=M)
        qkv = qkv.view(M, H + 2 * self.heads_kv, D)
        turned = qkv[:, :H + self.heads_kv]  # queries and keys, in place
        tq.rope(turned, pos, self.rope, Y=turned)
        tq.kv4_append(batch, qkv[:, H:H + self.heads_kv], qkv[:, H + self.heads_kv:])
        q = qkv[:, :H]
        tq.kv4_attention(batch, q, self.scale, self.workspace, O=q)
        return self.product("out", qkv.view(M, -1)[:, :H * D]), total

    def plain(self, x, residual, pos):
        """The same in fp32 for one sequence, nothing quantised."""
        import torch
        h = (x.float() + residual.float()).bfloat16().float()
        y = h * torch.rsqrt(h.pow(2).mean(-1, keepdim=True) + 1e-6) * self.gamma
        n, H, G, D = x.shape[0], self.heads, self.heads_kv, self.dim
        qkv = (y @ self.weights["qkv"][0].T).view(n, H + 2 * G, D)
        t = pos.float()[:, None, None] * self.inv_freq
        a, b = qkv[:, :H + G, :D // 2], qkv[:, :H + G, D // 2:]
        turned = torch.cat([a * t.cos() - b * t.sin(), a * t.sin() + b * t.cos()], -1)
        q, k, v = turned[:, :H], turned[:, H:], qkv[:, H + G:]
        k, v = (z.repeat_interleave(H // G, 1) for z in (k, v))
        s = torch.einsum("ihd,jhd->hij", q, k) * self.scale
        s.masked_fill_(torch.ones(n, n, device=s.device, dtype=torch.bool).triu(1), float("-inf"))
        return torch.einsum("hij,jhd->ihd", s.softmax(-1), v).reshape(n, H * D) @ self.weights["out"][0].T


def run(width=1024, heads=8, heads_kv=2, dim=128, lengths=(70, 1, 33, 200), steps=8, page=16, seed=0):
    """Prompts of the given lengths, then `steps` decoded tokens of each, the
    second step on captured as a graph.  Returns the layer's relative error
    against fp32 (prompts, decoded), the largest difference of a graph's step
    from the same step launched by itself, and a decoded step's time in us."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, total = len(lengths), sum(lengths)
    layer = Attention(width, heads, heads_kv, dim, seed=seed)
    cols = -(-(max(lengths) + steps) // page)
    cache = tq.KV4Cache(B * cols, page, heads_kv, dim)
    table = torch.randperm(B * cols, generator=g, device="cuda").int().view(B, cols)
    kv_len = torch.tensor(lengths, dtype=torch.int32, device="cuda")

    def rows(n):
        return (torch.randn(n, width, generator=g, device="cuda").bfloat16() for _ in range(2))

    starts = torch.tensor([0, *torch.tensor(lengths).cumsum(0)], dtype=torch.int32, device="cuda")
    prompts = tq.KV4Batch(cache, table, kv_len, starts, total, max(lengths))
    pos = torch.cat([torch.arange(n, device="cuda") for n in lengths]).int()[None]
    x, r = rows(total)
    out, _ = layer(x, r, prompts, pos)

    # decoding: the graph's own steps move the lengths on
    decode = tq.KV4Batch(cache, table, kv_len, torch.arange(B + 1, dtype=torch.int32, device="cuda"), B, 1)
    xs, rs = (torch.stack(z) for z in zip(*(tuple(rows(B)) for _ in range(steps))))
    at, step_x, step_r = kv_len[None].clone(), xs[0].clone(), rs[0].clone()
    outs = []

    def step():
        kv_len.add_(1)
        y, _ = layer(step_x, step_r, decode, at)
        at.add_(1)
        return y

    outs.append(step().clone())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    before = kv_len.clone(), at.clone()
    with torch.cuda.graph(graph):
        y = step()
    kv_len.copy_(before[0])
    at.copy_(before[1])
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    times, differ = [], 0.0
    for i in range(1, steps):
        step_x.copy_(xs[i])
        step_r.copy_(rs[i])
        begin.record()
        graph.replay()
        end.record()
        end.synchronize()
        times.append(1e3 * begin.elapsed_time(end))
        outs.append(y.clone())
        kv_len.sub_(1)                       # the same step once more, by itself
        at.sub_(1)
        differ = max(differ, float((step().float() - outs[-1].float()).abs().max()))
    if tq.device_status() != 0:
        raise RuntimeError("the device reported an error")

    num, den = [0.0, 0.0], [0.0, 0.0]
    for b, n in enumerate(lengths):
        s = int(starts[b])
        seq = torch.arange(n + steps, device="cuda")
        want = layer.plain(torch.cat([x[s:s + n], xs[:, b]]), torch.cat([r[s:s + n], rs[:, b]]), seq)
        got = torch.cat([out[s:s + n], torch.stack([o[b] for o in outs])]).float()
        for i, part in enumerate((slice(0, n), slice(n, None))):
            num[i] += float((got[part] - want[part]).pow(2).sum())
            den[i] += float(want[part].pow(2).sum())
    return [(a / b) ** 0.5 for a, b in zip(num, den)], differ, sorted(times)[len(times) // 2]


def main():
    a = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    for name, v in (("width", 4096), ("heads", 32), ("heads-kv", 8), ("dim", 128), ("batch", 16), ("prompt", 512),
                    ("steps", 16), ("page", 16)):
        a.add_argument("--" + name, type=int, default=v)
    a = a.parse_args()
    lengths = [1 + a.prompt * (i + 1) // a.batch for i in range(a.batch)]
    err, differ, us = run(a.width, a.heads, a.heads_kv, a.dim, lengths, a.steps, a.page)
    print(f"{a.batch} prompts of {lengths[0]} to {lengths[-1]} tokens, {a.steps} decoded tokens each")
    print(f"relative error against fp32: prompts {err[0]:.4f}, decoded {err[1]:.4f}")
    print(f"graph against single launches: {differ}")
    print(f"a decoded step of the layer: {us:.1f} us; a token's keys and values: "
          f"{a.heads_kv * (a.dim + 8)} bytes")


if __name__ == "__main__":
    main()
