"""A feed-forward layer of experts in 8-bit floating point, as measured cases: the
product of e4m3 operands with a scale for each block of 128, the experts'
feed-forward on rows sorted by expert, the router's choice with the sort it leads
to, and the weighted sum back into token order, with the gradients of the last two.

``run`` computes an operator in its plain form (elementary torch operations in
32 bits, rounded once at the end) or, where ``own`` is set, through the entry
points of ``dit_convrot_linear_gb300.tq``.  ``exact`` computes it in 64 bits.

Weights are codes and scales in the form in which models in this format are
published: any fp32 scale.  Activations are quantised within the pass, by scales
that are powers of two.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 128
MOST = 448.0                  # the largest e4m3 value


# ------------------------------------------------------------------- the cases

def listed():
    return [
        # one decoded token of the 896-wide decoder, gate or up projection: latency
        dict(name="product one token", op="product", rows=1, k=896, n=4864, out="bf16"),
        # a batch of decoded tokens of the 4096-wide decoder: the weights' stream
        dict(name="product batch", op="product", rows=48, k=4096, n=12288, out="bf16"),
        # a prompt of the 4096-wide decoder: the tensor cores
        dict(name="product prompt", op="product", rows=4032, k=4096, n=12288, out="bf16"),
        # no size a multiple of a tile, the last block of 128 not whole, fp32 out
        dict(name="product odd", op="product", rows=1013, k=2000, n=1100, out="f32"),
        # a batch of decoded tokens over 64 experts: most of them have a row or two
        dict(name="experts batch", op="experts", tokens=16, top=8, experts=64, width=2048, hidden=1024, skew=0.5,
             drop=0),
        # prompts over the same experts, some popular; an eighth of the choices lie elsewhere
        dict(name="experts prompt", op="experts", tokens=4096, top=8, experts=64, width=2048, hidden=1024, skew=1.0,
             drop=8),
        # the router of a decoded batch: latency
        dict(name="route batch", op="route", form="forward", tokens=16, experts=64, top=8, dtype="bf16", renorm=True,
             masked=0, idle=0),
        # the router of prompts with some experts out of reach and padding tokens
        dict(name="route prompt", op="route", form="forward", tokens=16384, experts=256, top=8, dtype="f32",
             renorm=True, masked=8, idle=100),
        # a training step's way back through the router
        dict(name="route gradient", op="route", form="gradient", tokens=16384, experts=256, top=8, dtype="f32",
             renorm=False, masked=0, idle=0),
        # the experts' rows of a decoded batch brought together: latency
        dict(name="combine batch", op="combine", form="forward", tokens=16, top=8, experts=64, width=2048, dtype="bf16",
             skew=0.5, drop=0),
        # the same of prompts of the 4096-wide decoder
        dict(name="combine prompt", op="combine", form="forward", tokens=8192, top=8, experts=64, width=4096,
             dtype="bf16", skew=1.0, drop=8),
        # a training step's way back: gradients of the rows and of the weights
        dict(name="combine gradient", op="combine", form="gradient", tokens=4096, top=8, experts=64, width=4096,
             dtype="bf16", skew=1.0, drop=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["product", "product", "experts", "experts", "route", "combine"])
    if op == "product":
        k = 16 * _log(rng, 4, 768)
        n = _log(rng, 64, 12288)
        rows = max(1, min(_log(rng, 1, 8192), 4032 * 4096 * 12288 // (k * n)))
        return dict(op=op, rows=rows, k=k, n=n, out=rng.choice(["bf16", "bf16", "f32"]))
    experts = _log(rng, 4, 256)
    top = rng.randint(1, min(8, experts))
    if op == "experts":
        width, hidden = 16 * _log(rng, 16, 256), 16 * _log(rng, 8, 128)
        experts = max(top, min(experts, 64 * 2048 * 1024 // (width * hidden)))
        tokens = max(1, min(_log(rng, 1, 8192), 32768 * 2048 * 1024 // (top * width * hidden)))
        return dict(op=op, tokens=tokens, top=top, experts=experts, width=width, hidden=hidden,
                    skew=rng.choice([0.0, 0.5, 1.0, 2.0]), drop=rng.choice([0, 0, 3, 8]))
    if op == "route":
        form = rng.choice(["forward", "forward", "gradient"])
        return dict(op=op, form=form, tokens=_log(rng, 1, 16384), experts=experts, top=top,
                    dtype=rng.choice(["bf16", "f32"]), renorm=rng.random() < 0.6,
                    masked=rng.choice([0, 0, rng.randint(0, experts - 1)]), idle=rng.choice([0, 0, 7]))
    form = rng.choice(["forward", "gradient"])
    width = 8 * _log(rng, 8, 1024)
    tokens = max(1, min(_log(rng, 1, 16384), (8192 if form == "forward" else 4096) * 8 * 4096 // (top * width) // 2))
    return dict(op=op, form=form, tokens=tokens, top=top, experts=experts, width=width,
                dtype=rng.choice(["bf16", "bf16", "f32"]), skew=rng.choice([0.0, 1.0]), drop=rng.choice([0, 3, 8]))


def _ceil(a, b):
    return -(-a // b)


def _size(t):
    return {"bf16": 2, "f32": 4}[t]


def _kept(c):
    """Choices that lead to a row (every drop-th one does not)."""
    n = c["tokens"] * c["top"]
    return n - (n // c["drop"] if c["drop"] else 0)


def work(c):
    if c["op"] == "product":
        m, n, k = c["rows"], c["n"], c["k"]
        return {"bytes": 2 * m * k + n * k + 4 * _ceil(n, BLOCK) * _ceil(k, BLOCK) + m * n * _size(c["out"]),
                "flops": 2 * m * n * k}
    t, top = c["tokens"], c["top"]
    if c["op"] == "experts":
        w, h, rows = c["width"], c["hidden"], _kept(c)
        active = c["experts"] * (1.0 - (1.0 - top / c["experts"]) ** t)     # of evenly popular experts
        return {"bytes": int(2 * t * w + active * 3 * w * h + 4 * rows + 2 * rows * w), "flops": 6 * rows * w * h}
    if c["op"] == "route":
        e, size = c["experts"], _size(c["dtype"])
        if c["form"] == "forward":      # the choice is written, read by the sort, and its three lists written
            return {"bytes": t * e * size + 20 * t * top + 4 * e, "flops": 4 * t * e}
        return {"bytes": 2 * t * e * size + 8 * t * top, "flops": 6 * t * e}
    w, rows, size = c["width"], _kept(c), _size(c["dtype"])
    if c["form"] == "forward":
        return {"bytes": size * (rows + t) * w + 8 * t * top, "flops": 2 * rows * w}
    return {"bytes": size * (2 * rows + t) * w + 12 * t * top, "flops": 3 * rows * w}


# ------------------------------------------------------------------ the inputs

def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _outliers(x, g):
    """A few channels forty times the others, as a residual stream has them."""
    n = x.shape[-1]
    k = max(1, n // 500)
    x[..., torch.randint(0, n, (k,), generator=g, device=DEV)] *= 40.0
    return x


def _weights(g, n, k):
    """A published matrix: e4m3 codes (as bytes) and a scale amax / 448 for each
    block of 128 rows and 128 columns."""
    nb, kb = _ceil(n, BLOCK), _ceil(k, BLOCK)
    w = torch.zeros(nb * BLOCK, kb * BLOCK, device=DEV)
    w[:n, :k] = _normal(g, n, k) / math.sqrt(k)
    b = w.view(nb, BLOCK, kb, BLOCK)
    s = b.abs().amax((1, 3)) / MOST
    codes = (b / s[:, None, :, None]).clamp(-MOST, MOST).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes.view(nb * BLOCK, kb * BLOCK)[:n, :k].contiguous(), s


def _choices(g, c):
    """Each token's experts, int32 [tokens, top]; every drop-th choice is none."""
    t, e = c["tokens"], c["experts"]
    popular = c["skew"] * torch.cos(torch.arange(e, device=DEV) * 2.4)
    ids = (_normal(g, t, e) + popular).argsort(1, descending=True)[:, :c["top"]].int().contiguous()
    if c["drop"]:
        flat = ids.view(-1)
        flat[c["drop"] - 1::c["drop"]] = -1
    return ids


def _sorted(ids, experts):
    """Offsets, token of each sorted row, place of each choice (as lists of the sort)."""
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < experts), flat, experts)
    order = torch.argsort(key, stable=True)
    count = torch.zeros(experts + 1, dtype=torch.int64, device=DEV).scatter_add_(0, key, torch.ones_like(key))
    offsets = torch.nn.functional.pad(count[:experts].cumsum(0), (1, 0))
    at = torch.arange(flat.numel(), device=DEV)
    used = at < offsets[-1]
    token = torch.where(used, order // ids.shape[1], -1)
    place = torch.full_like(flat, -1).scatter_(0, order, torch.where(used, at, -1))
    return offsets.int(), token.int(), place.view(ids.shape).int()


def _type(t):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[t]


def prepare(case, seed):
    c = dict(case)
    g = _generator(seed)
    s = {"case": c}
    if c["op"] == "product":
        s["x"] = _outliers(_normal(g, c["rows"], c["k"]), g).bfloat16()
        s["w"], s["sw"] = _weights(g, c["n"], c["k"])
        if own:
            from dit_convrot_linear_gb300 import tq
            s["y"] = torch.empty(c["rows"], c["n"], dtype=_type(c["out"]), device=DEV)
            s["q"] = torch.empty(c["rows"], c["k"], dtype=torch.uint8, device=DEV)
            s["sx"] = torch.empty(_ceil(c["k"], BLOCK), c["rows"], device=DEV)
            s["work"] = tq.f8_workspace()
        return s
    if c["op"] == "experts":
        w, h, e = c["width"], c["hidden"], c["experts"]
        rows = c["tokens"] * c["top"]
        s["x"] = _outliers(_normal(g, c["tokens"], w), g).bfloat16()
        s["offsets"], s["token"], _ = _sorted(_choices(g, c), e)
        for name, n, k in (("up", 2 * h, w), ("down", w, h)):
            codes = torch.empty(e, n, k, dtype=torch.uint8, device=DEV)
            scales = torch.empty(e, _ceil(n, BLOCK), _ceil(k, BLOCK), device=DEV)
            for i in range(e):
                codes[i], scales[i] = _weights(g, n, k)
            s[name], s["s" + name] = codes, scales
        s["y"] = torch.zeros(rows, w, dtype=torch.bfloat16, device=DEV)     # rows past the last expert's stay
        if own:
            from dit_convrot_linear_gb300 import tq
            s["gu"] = torch.zeros(rows, 2 * h, dtype=torch.bfloat16, device=DEV)
            s["xq"] = torch.empty(rows, w, dtype=torch.uint8, device=DEV)
            s["hq"] = torch.empty(rows, h, dtype=torch.uint8, device=DEV)
            s["sx"] = torch.empty(_ceil(w, BLOCK), rows, device=DEV)
            s["sh"] = torch.empty(_ceil(h, BLOCK), rows, device=DEV)
            s["work"] = tq.f8_workspace()
        else:
            s["ends"] = s["offsets"].tolist()      # the plain form launches by the host's counts
        return s
    if c["op"] == "route":
        t, e = c["tokens"], c["experts"]
        x = _normal(g, t, e) * 1.5
        if c["masked"]:                            # as many experts out of a token's reach
            x = x.masked_fill(torch.rand(t, e, generator=g, device=DEV).argsort(1) < c["masked"], -math.inf)
        if c["idle"]:                              # padding tokens choose none
            x[c["idle"] - 1::c["idle"]] = -math.inf
        s["x"] = x.to(_type(c["dtype"]))
        if c["form"] == "gradient":
            s["ids"] = _plain_choice(s["x"], c["top"])[0]
            s["dw"] = _normal(g, t, c["top"])
            s["dx"] = torch.empty_like(s["x"])
        elif own:
            i32 = dict(dtype=torch.int32, device=DEV)
            s["ids"] = torch.empty(t, c["top"], **i32)
            s["weights"] = torch.empty(t, c["top"], device=DEV)
            s["lists"] = (torch.empty(e + 1, **i32), torch.empty(t * c["top"], **i32),
                          torch.empty(t, c["top"], **i32))
        return s
    t, top, w = c["tokens"], c["top"], c["width"]
    _, _, s["place"] = _sorted(_choices(g, c), c["experts"])
    s["weights"] = torch.softmax(_normal(g, t, top), -1)
    s["y"] = _normal(g, t * top, w).to(_type(c["dtype"]))
    if c["form"] == "forward":
        s["out"] = torch.empty(t, w, dtype=_type(c["dtype"]), device=DEV)
    else:
        s["do"] = _normal(g, t, w).to(_type(c["dtype"]))
        # rows past the last expert's stay; one more, where a choice that leads to no row writes
        s["dy"] = torch.zeros(t * top + 1, w, dtype=_type(c["dtype"]), device=DEV)
        s["dw"] = torch.empty(t, top, device=DEV)
    return s


# --------------------------------------------------------------------- one pass

def run(s):
    c = s["case"]
    return (_own if own else _plain)[c["op"], c.get("form")](s)


def _own_product(s):
    from dit_convrot_linear_gb300 import tq
    q, sx = tq.quant_act_f8(s["x"], Xq=s["q"], sx=s["sx"])
    return tq.linear_f8(q, sx, s["w"], s["sw"], s["work"], out=s["case"]["out"], Y=s["y"])


def _own_experts(s):
    from dit_convrot_linear_gb300 import tq
    h = s["case"]["hidden"]
    q, sx = tq.quant_act_f8(s["x"], rows=s["token"], Xq=s["xq"], sx=s["sx"])
    gu = tq.linear_f8_experts(q, sx, s["offsets"], s["up"], s["sup"], s["work"], out="bf16", Y=s["gu"])
    q, sh = tq.swiglu_quant_act_f8(gu[:, :h], gu[:, h:], Xq=s["hq"], sx=s["sh"])
    return tq.linear_f8_experts(q, sh, s["offsets"], s["down"], s["sdown"], s["work"], out="bf16", Y=s["y"])


def _own_route(s):
    from dit_convrot_linear_gb300 import tq
    c = s["case"]
    ids, w = tq.expert_topk(s["x"], c["top"], renorm=c["renorm"], ids=s["ids"], weights=s["weights"])
    offsets, token, place = tq.expert_sort(ids, c["experts"], *s["lists"])
    return dict(ids=ids, weights=w, offsets=offsets, token=token, place=place)


def _own_route_gradient(s):
    from dit_convrot_linear_gb300 import tq
    return tq.expert_topk_grad(s["x"], s["ids"], s["dw"], renorm=s["case"]["renorm"], dlogits=s["dx"])


def _own_combine(s):
    from dit_convrot_linear_gb300 import tq
    return tq.expert_combine(s["y"], s["place"], s["weights"], O=s["out"])


def _own_combine_gradient(s):
    from dit_convrot_linear_gb300 import tq
    return tq.expert_combine_grad(s["do"], s["y"], s["place"], s["weights"], dY=s["dy"][:-1], dweights=s["dw"])


def _quantised(x):
    """Rows rounded to e4m3 by blocks of 128 columns with power-of-two scales, as
    the values their codes stand for (fp32)."""
    m, k = x.shape
    b = torch.nn.functional.pad(x, (0, -k % BLOCK)).view(m, -1, BLOCK)
    part, power = torch.frexp(b.abs().amax(-1, keepdim=True))          # part in [1/2, 1)
    power = (power - 9 + (part > 0.875).int()).clamp(min=-126)
    s = ((power + 127) << 23).view(torch.float32)
    return ((b / s).to(torch.float8_e4m3fn).float() * s).view(m, -1)[:, :k]


def _dequantised(codes, scales):
    n, k = codes.shape
    s = scales.repeat_interleave(BLOCK, 0)[:n].repeat_interleave(BLOCK, 1)[:, :k]
    return codes.view(torch.float8_e4m3fn).float() * s


def _plain_product(s):
    x = _quantised(s["x"].float())
    return torch.matmul(x, _dequantised(s["w"], s["sw"]).t()).to(_type(s["case"]["out"]))


def _plain_experts(s):
    c, y = s["case"], s["y"]
    h, ends = c["hidden"], s["ends"]
    x = _quantised(s["x"].float())
    for e in range(c["experts"]):
        a, b = ends[e], ends[e + 1]
        if a == b:
            continue
        rows = x[s["token"][a:b].long()]
        gu = torch.matmul(rows, _dequantised(s["up"][e], s["sup"][e]).t()).bfloat16().float()
        g, u = gu[:, :h], gu[:, h:]
        z = _quantised(g / (1.0 + torch.exp(-g)) * u)
        y[a:b] = torch.matmul(z, _dequantised(s["down"][e], s["sdown"][e]).t()).bfloat16()
    return y


def _plain_choice(x, top):
    x = x.float()
    v, ids = torch.sort(x, dim=1, descending=True, stable=True)
    v, ids = v[:, :top], ids[:, :top]
    return torch.where(v > -math.inf, ids, -1).int().contiguous(), v


def _softmax(x):
    x = x.float()
    m = x.amax(1, keepdim=True)
    p = torch.exp(x - torch.where(m > -math.inf, m, 0.0))
    total = p.sum(1, keepdim=True)
    return p / torch.where(total > 0, total, 1.0)


def _plain_route(s):
    c = s["case"]
    ids, _ = _plain_choice(s["x"], c["top"])
    w = torch.where(ids >= 0, torch.gather(_softmax(s["x"]), 1, ids.clamp(min=0).long()), 0.0)
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = w / torch.where(total > 0, total, 1.0)
    offsets, token, place = _sorted(ids, c["experts"])
    return dict(ids=ids, weights=w, offsets=offsets, token=token, place=place)


def _plain_route_gradient(s):
    c, x = s["case"], s["x"].float()
    chosen = s["ids"] >= 0
    ids = s["ids"].clamp(min=0).long()
    dw = torch.where(chosen, s["dw"], 0.0)
    p = _softmax(x)
    if c["renorm"]:
        w = torch.where(chosen, torch.gather(p, 1, ids), 0.0)
        total = w.sum(1, keepdim=True)
        w = w / torch.where(total > 0, total, 1.0)
        part = w * (dw - (w * dw).sum(1, keepdim=True))
        return torch.zeros_like(x).scatter_add_(1, ids, part).to(s["x"].dtype)
    d = torch.zeros_like(x).scatter_add_(1, ids, dw)
    return (p * (d - (p * d).sum(1, keepdim=True))).to(s["x"].dtype)


def _plain_combine(s):
    out = torch.zeros(s["case"]["tokens"], s["case"]["width"], device=DEV)
    for j in range(s["case"]["top"]):
        at = s["place"][:, j].long()
        row = s["y"][at.clamp(min=0)].float() * s["weights"][:, j, None]
        out += torch.where(at[:, None] >= 0, row, 0.0)
    return out.to(s["y"].dtype)


def _plain_combine_gradient(s):
    do = s["do"].float()
    dw = []
    for j in range(s["case"]["top"]):
        at = s["place"][:, j].long()
        keep = at >= 0
        dw.append(torch.where(keep, (s["y"][at.clamp(min=0)].float() * do).sum(1), 0.0))
        s["dy"][torch.where(keep, at, s["y"].shape[0])] = (do * s["weights"][:, j, None]).to(s["y"].dtype)
    return s["dy"][:-1], torch.stack(dw, 1)


_plain = {("product", None): _plain_product, ("experts", None): _plain_experts, ("route", "forward"): _plain_route,
          ("route", "gradient"): _plain_route_gradient, ("combine", "forward"): _plain_combine,
          ("combine", "gradient"): _plain_combine_gradient}
_own = {("product", None): _own_product, ("experts", None): _own_experts, ("route", "forward"): _own_route,
        ("route", "gradient"): _own_route_gradient, ("combine", "forward"): _own_combine,
        ("combine", "gradient"): _own_combine_gradient}


# ------------------------------------------------------------- in 64 bits

def _e4m3(v):
    """The nearest e4m3 value (ties to the even code): steps of an eighth of the
    value's power of two, 2^-9 below 2^-6."""
    power = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(power - 3.0)
    return torch.round(v / step) * step


def _exact_rows(x):
    """[blocks of 128 columns of x, 64 bits] as quantised values."""
    out = torch.empty_like(x)
    for b in range(0, x.shape[1], BLOCK):
        v = x[:, b:b + BLOCK]
        a = v.abs().max(1, keepdim=True).values
        power = torch.ceil(torch.log2((a / MOST).clamp(min=2.0 ** -126)))
        power = torch.where(MOST * torch.exp2(power - 1.0) >= a, power - 1.0, power)   # log2's own rounding
        power = torch.where(MOST * torch.exp2(power) < a, power + 1.0, power)
        s = torch.exp2(power.clamp(min=-126.0))
        out[:, b:b + BLOCK] = _e4m3(v / s) * s
    return out


def _exact_matrix(codes, scales):
    """Codes by their bits: sign, four bits of exponent, three of mantissa."""
    c = codes.int()
    e, m = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e > 0, (8.0 + m) * torch.exp2((e - 10).double()), m * 2.0 ** -9)
    v = torch.where(c >= 128, -v, v)
    for i in range(scales.shape[0]):
        for j in range(scales.shape[1]):
            v[i * BLOCK:(i + 1) * BLOCK, j * BLOCK:(j + 1) * BLOCK] *= scales[i, j].double()
    return v


def exact(case, seed):
    s = prepare(case, seed)
    return {"product": _exact_product, "experts": _exact_experts, "route": _exact_route,
            "combine": _exact_combine}[case["op"]](s)


def _exact_product(s):
    return _exact_rows(s["x"].double()) @ _exact_matrix(s["w"], s["sw"]).t()


def _exact_experts(s):
    c = s["case"]
    h, ends = c["hidden"], s["offsets"].tolist()
    y = torch.zeros(s["y"].shape, dtype=torch.float64, device=DEV)
    x = _exact_rows(s["x"].double())
    for e in range(c["experts"]):
        a, b = ends[e], ends[e + 1]
        if a == b:
            continue
        gu = x[s["token"][a:b].long()] @ _exact_matrix(s["up"][e], s["sup"][e]).t()
        gu = gu.bfloat16().double()                # the projection's output is stored in bf16
        g, u = gu[:, :h], gu[:, h:]
        y[a:b] = _exact_rows(torch.sigmoid(g) * g * u) @ _exact_matrix(s["down"][e], s["sdown"][e]).t()
    return y


def _exact_route(s):
    c, x = s["case"], s["x"].double()
    p = torch.softmax(x, 1).nan_to_num(0.0)        # a row without any expert has no probabilities
    if c["form"] == "gradient":
        x = x.clone().requires_grad_(True)
        chosen = s["ids"] >= 0
        v = torch.where(chosen, torch.gather(x, 1, s["ids"].clamp(min=0).long()), -math.inf)
        if c["renorm"]:
            some = chosen.any(1, keepdim=True)
            w = torch.softmax(torch.where(some, v, 0.0), 1)
        else:
            some = chosen.any(1, keepdim=True)
            top = torch.where(some, x.detach().max(1, keepdim=True).values, 0.0)
            w = torch.exp(v - top) / torch.where(some, torch.exp(x - top).sum(1, keepdim=True), 1.0)
        total = (torch.where(chosen & some, w, 0.0) * s["dw"].double()).sum()
        return torch.autograd.grad(total, x)[0].nan_to_num(0.0)
    order = torch.argsort(-x, dim=1, stable=True)[:, :c["top"]]
    chosen = torch.gather(x, 1, order) > -math.inf
    ids = torch.where(chosen, order, -1)
    w = torch.gather(p, 1, order) * chosen
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    # the sort, from counts alone
    flat = ids.reshape(-1)
    hits = torch.zeros(flat.numel(), c["experts"], dtype=torch.int32, device=DEV)
    rows = torch.nonzero(flat >= 0).squeeze(1)
    hits[rows, flat[rows]] = 1
    before = hits.cumsum(0, dtype=torch.int32)
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), hits.sum(0).cumsum(0)])
    place = torch.full_like(flat, -1)
    place[rows] = offsets[flat[rows]] + before[rows, flat[rows]] - 1
    token = torch.full_like(flat, -1)
    token[place[rows]] = rows // c["top"]
    return dict(ids=ids.int(), weights=w, offsets=offsets.int(), token=token.int(),
                place=place.view(ids.shape).int())


def _exact_combine(s):
    c = s["case"]
    place, w = s["place"].long(), s["weights"].double()
    if c["form"] == "forward":
        out = torch.zeros(c["tokens"], c["width"], dtype=torch.float64, device=DEV)
        for j in range(c["top"]):
            t = torch.nonzero(place[:, j] >= 0).squeeze(1)
            out[t] += w[t, j, None] * s["y"][place[t, j]].double()
        return out
    dy = torch.zeros(s["y"].shape, dtype=torch.float64, device=DEV)
    dw = torch.zeros(c["tokens"], c["top"], dtype=torch.float64, device=DEV)
    for j in range(c["top"]):
        t = torch.nonzero(place[:, j] >= 0).squeeze(1)
        do = s["do"][t].double()
        dy[place[t, j]] = w[t, j, None] * do
        dw[t, j] = torch.einsum("tw,tw->t", do, s["y"][place[t, j]].double())
    return dy, dw
