"""The router, the sort by expert and the rows there and back, against 64 bits.

Bars, set before the first run:
  - ids, offsets, tokens, places and gathered rows are equal;
  - the router's weights: an exponential of at most 2 ulp (2^-22) on each side of a
    quotient of sums of up to 1024 terms (ten levels of 2^-24 in trees, up to 32 in
    the lanes' own chains), its argument's rounding (2^-24 of |x - max|, which moves
    the exponential by as much): (2^-20 + 2^-23 |x - max|) of the weight;
  - its gradients: the same of the sum of their terms' magnitudes, with the sum's
    32 roundings: 2^-18 (1 + span / 8) of it; half a step of bf16 (2^-8) on top there;
  - sums of rows: `top` fmas of 2^-24 each of the terms' magnitudes, and half a step
    of the output (2^-8 for bf16);
  - products of a row with a row: fma chains of at most width / 256 + 8, then 5 and 3
    levels: (width / 256 + 24) 2^-24 of the terms' magnitudes.
"""
import math

import pytest

import f8_ref as ref

pytestmark = pytest.mark.gpu

DTYPES = ["float32", "bfloat16"]


def gen(seed):
    import torch
    return torch.Generator(device="cuda").manual_seed(seed)


def logits(g, T, E, dtype, masked=0, pad=0):
    import torch
    x = 2.0 * torch.randn(T, E + pad, generator=g, device="cuda")
    x = torch.round(x * 8) / 8                  # equal ones among them
    if masked:
        x[:, :E].masked_fill_(torch.rand(T, E, generator=g, device="cuda").argsort(1) < masked, -math.inf)
    if T > 4:
        x[T // 2] = -math.inf                   # a padding token
        x[T // 3] = 1.0                         # all equal
    return x.to(getattr(torch, dtype))[:, :E]


ROUTES = [(1, 1, 1, 0), (1, 64, 8, 0), (5, 3, 2, 1), (40, 8, 8, 3), (33, 60, 6, 0), (17, 64, 8, 60), (200, 128, 4, 0),
          (65, 129, 32, 0), (64, 256, 8, 8), (9, 500, 2, 0), (20, 1000, 32, 990), (7, 1024, 16, 0)]


def bar_weights(x, ids, w):
    import torch
    m = x.double().max(1, keepdim=True).values
    span = (torch.where(torch.isfinite(m), m, 0.0) - torch.gather(x.double(), 1, ids.clamp(min=0).long())).abs()
    return w * (2.0 ** -20 + 2.0 ** -23 * torch.where(ids >= 0, span, 0.0))


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,E,top,masked", ROUTES)
def test_topk(tq, T, E, top, masked, dtype, renorm):
    import torch
    x = logits(gen(T + E), T, E, dtype, masked, T % 3)
    ids, w = tq.expert_topk(x, top, renorm=renorm)
    assert torch.equal(ids.cpu(), ref.topk(x, top))
    want = ref.weights(x, ids, renorm)
    assert ((w.double() - want).abs() <= bar_weights(x, ids, want)).all()
    assert (w[ids < 0] == 0).all()
    a, b = tq.expert_topk(x, top, renorm=renorm)
    assert torch.equal(a, ids) and torch.equal(b, w)


@pytest.mark.parametrize("top", [1, 2, 8, 9, 32])
def test_topk_many_near_the_last(tq, top):
    """Rows in which more or fewer reach the last choice than a warp has lanes: equal
    ones among them, the large ones in one lane's column or one after the other, NaN."""
    import torch
    E = 256
    g = gen(top)
    x = torch.randn(12, E, generator=g, device="cuda")
    for i, n in enumerate((1, 31, 32, 33, 64)):
        at = torch.randperm(E, generator=g, device="cuda")[:n]
        x[i, at] = 5.0
    x[5, ::32] = torch.arange(8.0, device="cuda") + 4      # one lane's
    x[6] = torch.arange(E, device="cuda") / 8.0
    x[7] = -x[6]
    x[8, ::2] = math.nan
    x[9] = -math.inf
    x[9, 255] = -1.0
    x[10, 40:] = -math.inf
    x[11, 77] = math.inf
    ids, w = tq.expert_topk(x, top)
    assert torch.equal(ids.cpu(), ref.topk(x, top))
    fine = [i for i in range(12) if i not in (8, 11)]
    want = ref.weights(x[fine], ids[fine], True)
    assert ((w[fine].double() - want).abs() <= bar_weights(x[fine], ids[fine], want)).all()
    assert torch.isnan(w[[8, 11]]).any(1).all()


@pytest.mark.parametrize("renorm", [True, False])
def test_topk_not_finite(tq, renorm):
    import torch
    x = torch.tensor([[0.0, math.nan, 3.0, 1.0], [math.inf, 0.0, -math.inf, 2.0], [1e30, -1e30, 3e38, -3e38],
                      [-math.nan, math.nan, 5.0, math.inf], [-0.0, 0.0, -0.0, 0.0]], device="cuda")
    ids, w = tq.expert_topk(x, 3, renorm=renorm)
    assert ids.cpu().tolist() == [[1, 2, 3], [0, 3, 1], [2, 0, 1], [0, 1, 3], [0, 1, 2]]
    assert torch.isnan(w[[0, 1, 3]]).any(1).all() and not torch.isnan(w[[2, 4]]).any()
    assert w[2].tolist() == [1.0, 0.0, 0.0]


def exact_grad(x, ids, dw, renorm):
    """(dlogits, the sum of each one's terms' magnitudes) from the formula."""
    import torch
    x, dw, ids = x.double(), dw.double(), ids.long()
    at = ids.clamp(min=0)
    keep = ids >= 0
    dw = torch.where(keep, dw, 0.0)
    m = x.max(1, keepdim=True).values
    p = torch.exp(x - torch.where(torch.isfinite(m), m, 0.0))
    if renorm:
        w = torch.where(keep, torch.gather(p, 1, at), 0.0)
        t = w.sum(1, keepdim=True)
        w = w / torch.where(t > 0, t, 1.0)
        mean = (w * dw).sum(1, keepdim=True)
        size = w * (dw.abs() + (w * dw.abs()).sum(1, keepdim=True))
        return torch.zeros_like(x).scatter_add_(1, at, w * (dw - mean)), torch.zeros_like(x).scatter_add_(1, at, size)
    t = p.sum(1, keepdim=True)
    p = p / torch.where(t > 0, t, 1.0)
    d = torch.zeros_like(x).scatter_add_(1, at, dw)
    a = torch.zeros_like(x).scatter_add_(1, at, dw.abs())
    return p * (d - (p * d).sum(1, keepdim=True)), p * (a + (p * a).sum(1, keepdim=True))


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,E,top,masked", ROUTES)
def test_topk_grad(tq, T, E, top, masked, dtype, renorm):
    import torch
    g = gen(T)
    x = logits(g, T, E, dtype, masked, T % 2)
    ids, _ = tq.expert_topk(x, top, renorm=renorm)
    dw = torch.randn(T, top, generator=g, device="cuda")
    dx = tq.expert_topk_grad(x, ids, dw, renorm=renorm)
    want, size = exact_grad(x, ids, dw, renorm)
    bar = size * 2.0 ** -18 * 3 + (want.abs() * 2.0 ** -8 if dtype == "bfloat16" else 0.0)
    assert ((dx.double() - want).abs() <= bar + 1e-40).all()


@pytest.mark.parametrize("renorm", [True, False])
def test_topk_grad_is_the_slope(tq, renorm):
    """Against differences of the 64-bit weights, the choice held."""
    import torch
    g = gen(3)
    x = logits(g, 6, 20, "float32")
    ids, _ = tq.expert_topk(x, 4, renorm=renorm)
    dw = torch.randn(6, 4, generator=g, device="cuda")
    dx = tq.expert_topk_grad(x, ids, dw, renorm=renorm)
    h = 1e-5
    for e in range(20):
        up, down = x.double(), x.double()
        up[:, e] += h
        down[:, e] -= h
        slope = ((ref.weights(up, ids, renorm) - ref.weights(down, ids, renorm)) * dw.double()).sum(1) / (2 * h)
        assert ((dx[:, e].double() - slope).abs() <= 1e-6).all()


def test_topk_grad_choices_twice_and_out_of_range(tq):
    """A choice named twice counts twice; ids out of range count for nothing and are
    reported."""
    import torch
    x = logits(gen(4), 3, 9, "float32")
    dw = torch.tensor([[1.0, 2.0, -1.0], [0.5, 0.25, 4.0], [1.0, 1.0, 1.0]], device="cuda")
    ids = torch.tensor([[2, 2, 5], [8, 0, 8], [1, -1, 1]], dtype=torch.int32, device="cuda")
    for renorm in (True, False):
        want, size = exact_grad(x, ids, dw, renorm)
        got = tq.expert_topk_grad(x, ids, dw, renorm=renorm)
        assert ((got.double() - want).abs() <= size * 2.0 ** -17).all()
        assert tq.device_status() == 0
        bad = torch.where(ids == 8, 9, ids)
        got = tq.expert_topk_grad(x, bad, dw, renorm=renorm)
        want, size = exact_grad(x, torch.where(ids == 8, -1, ids), dw, renorm)
        assert ((got.double() - want).abs() <= size * 2.0 ** -17).all()
        assert tq.device_status() == 11


# ------------------------------------------------------------------- the sort

def choices(g, T, top, E, drop=0.0, skew=False):
    import torch
    r = torch.rand(T, top, generator=g, device="cuda")
    ids = ((r * r * r if skew else r) * E).int().clamp(max=E - 1)
    return torch.where(torch.rand(T, top, generator=g, device="cuda") < drop, -1, ids).int()


SORTS = [(1, 1, 1, 0.0), (1, 8, 64, 0.0), (3, 2, 2, 0.5), (16, 8, 64, 0.0), (100, 1, 7, 0.1), (33, 31, 1, 0.0),
         (300, 8, 1024, 0.2), (1000, 6, 60, 0.0), (50, 4, 8, 1.0), (4099, 8, 256, 0.1), (5000, 32, 33, 0.0)]


@pytest.mark.parametrize("skew", [False, True])
@pytest.mark.parametrize("T,top,E,drop", SORTS)
def test_sort(tq, T, top, E, drop, skew):
    import torch
    ids = choices(gen(T), T, top, E, drop, skew)
    off, token, place = tq.expert_sort(ids, E)
    # against the stable sort of (expert, position)
    flat = ids.reshape(-1).long().cpu()
    key = torch.where(flat >= 0, flat, E)
    order = torch.argsort(key, stable=True)
    n = int((flat >= 0).sum())
    assert off.cpu().tolist() == [0, *torch.bincount(key, minlength=E + 1)[:E].cumsum(0).tolist()]
    assert torch.equal(token.cpu().long(), torch.cat([order[:n] // top, torch.full((flat.numel() - n,), -1)]))
    back = torch.full_like(flat, -1)
    back[order[:n]] = torch.arange(n)
    assert torch.equal(place.cpu().reshape(-1).long(), back)
    assert tq.device_status() == 0
    if flat.numel() < 300:
        want = ref.sort(ids.cpu(), E)
        assert all(torch.equal(a.cpu(), b) for a, b in zip((off, token, place), want))


@pytest.mark.parametrize("T,top,E,drop", [(400, 8, 1000, 0.3), (700, 4, 33, 1.0), (1025, 2, 1, 0.97), (2081, 1, 1023, 0.0)])
def test_sort_whose_lanes_part(tq, T, top, E, drop):
    """Clusters whose warps' lanes leave the loops over experts, choices and the rows behind
    the last one at different times, twenty times each."""
    import torch
    ids = choices(gen(E), T, top, E, drop)
    flat = ids.reshape(-1).long().cpu()
    n = int((flat >= 0).sum())
    order = torch.argsort(torch.where(flat >= 0, flat, E), stable=True)
    want = torch.cat([order[:n] // top, torch.full((flat.numel() - n,), -1)]).int()
    got = [tq.expert_sort(ids, E) for _ in range(20)]
    for off, token, place in got:
        assert torch.equal(token.cpu(), want)
        assert all(torch.equal(a, b) for a, b in zip((off, place), (got[0][0], got[0][2])))
    assert int(got[0][0][E]) == n
    assert tq.device_status() == 0


def test_sort_many(tq):
    """Half a million choices and more, one expert's share past 65536."""
    import torch
    ids = choices(gen(1), 90001, 8, 16, 0.05, True)
    off, token, place = tq.expert_sort(ids, 16)
    flat = ids.reshape(-1).long()
    key = torch.where(flat >= 0, flat, 16)
    order = torch.argsort(key, stable=True)
    n = int((flat >= 0).sum())
    assert int(off[-1]) == n and torch.equal(token[:n].long(), order[:n] // 8) and (token[n:] == -1).all()
    assert torch.equal(place.reshape(-1)[order[:n]].long(), torch.arange(n, device="cuda"))
    assert (place[ids < 0] == -1).all()


def test_sort_without_tokens_and_out_of_range(tq):
    import torch
    off, token, place = tq.expert_sort(torch.empty(0, 2, dtype=torch.int32, device="cuda"), 5)
    assert off.tolist() == [0] * 6
    off, token, place = tq.expert_sort(torch.tensor([[0, 5], [-7, 4], [-1, 0]], dtype=torch.int32, device="cuda"), 5)
    assert tq.device_status() == 11
    assert off.tolist() == [0, 2, 2, 2, 2, 3] and token.tolist() == [0, 2, 1, -1, -1, -1]
    assert place.tolist() == [[0, -1], [-1, 2], [-1, 1]]


# ------------------------------------------------------------ rows there and back

ROWS = [(1, 1, 1, 8), (16, 8, 64, 2048), (5, 3, 4, 24), (300, 6, 60, 896), (70, 2, 8, 4096), (9, 32, 64, 520),
        (2, 8, 16, 16384)]


def case(tq, T, top, E, W, dtype, pad=0):
    import torch
    g = gen(T + W)
    ids = choices(g, T, top, E, 0.15)
    _, token, place = tq.expert_sort(ids, E)
    y = torch.randn(T * top, W + pad, generator=g, device="cuda").to(getattr(torch, dtype))[:, :W]
    w = torch.rand(T, top, generator=g, device="cuda")
    return g, token, place, y, w


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,top,E,W", ROWS)
def test_gather(tq, T, top, E, W, dtype):
    import torch
    g, token, _, _, _ = case(tq, T, top, E, W, dtype)
    x = torch.randn(T, W + 8, generator=g, device="cuda").to(getattr(torch, dtype))[:, :W]
    y = torch.full((T * top, W), 3.0, dtype=x.dtype, device="cuda")
    tq.expert_gather(x, token, Y=y)
    assert torch.equal(y, torch.where((token >= 0)[:, None], x[token.clamp(min=0).long()], 3.0))
    bad = torch.where(token == 0, T, token)
    if (bad == T).any():
        tq.device_status()
        tq.expert_gather(x, bad, Y=y.fill_(3.0))
        assert tq.device_status() == 11 and (y[bad == T] == 3.0).all()


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,top,E,W", ROWS)
def test_combine(tq, T, top, E, W, dtype, weighted):
    import torch
    _, _, place, y, w = case(tq, T, top, E, W, dtype, 8)
    frame = torch.full((T + 2, W + 16), 3.0, dtype=y.dtype, device="cuda")
    O = frame[1:T + 1, 8:W + 8] if dtype == "bfloat16" else frame[1:T + 1, 4:W + 4]
    tq.expert_combine(y, place, w if weighted else None, O=O)
    at = place.long().clamp(min=0)
    c = torch.where(place >= 0, w.double() if weighted else 1.0, 0.0)
    terms = c[:, :, None] * y.double()[at]
    want, size = terms.sum(1), terms.abs().sum(1)
    bar = size * top * 2.0 ** -24 + (want.abs() * 2.0 ** -8 if dtype == "bfloat16" else 0.0) * 1.01
    assert ((O.double() - want).abs() <= bar).all()
    frame[1:T + 1, 8 if dtype == "bfloat16" else 4:][:, :W] = 3.0
    assert (frame == 3.0).all()
    assert (O == 3.0).all()


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,top,E,W", ROWS)
def test_combine_grad(tq, T, top, E, W, dtype, weighted):
    import torch
    g, _, place, y, w = case(tq, T, top, E, W, dtype, 8)
    dO = torch.randn(T, W + 16, generator=g, device="cuda").to(y.dtype)[:, :W]
    dY = torch.full((T * top, W), 3.0, dtype=y.dtype, device="cuda")
    _, dw = tq.expert_combine_grad(dO, y, place, w if weighted else None, dY=dY)
    keep = place >= 0
    want = torch.full((T * top, W), 3.0, dtype=torch.float64, device="cuda")
    c = w.double() if weighted else torch.ones_like(w).double()
    want[place[keep].long()] = (c[:, :, None] * dO.double()[:, None])[keep]
    half = 2.0 ** -8 if dtype == "bfloat16" else 2.0 ** -24
    assert ((dY.double() - want).abs() <= want.abs() * half * 1.01).all()
    terms = y.double()[place.long().clamp(min=0)] * dO.double()[:, None]
    exact = torch.where(keep, terms.sum(2), 0.0)
    assert ((dw.double() - exact).abs() <= terms.abs().sum(2) * (W / 256 + 24) * 2.0 ** -24).all()
    assert (dw[~keep] == 0).all()
    again, dw2 = tq.expert_combine_grad(dO, y, place, w if weighted else None, dY=torch.full_like(dY, 3.0))
    assert torch.equal(again, dY) and torch.equal(dw2, dw)


def test_combine_grad_is_the_slope(tq):
    """dO . (combine at w + h - combine at w - h), and the same along a row of Y."""
    import torch
    g, _, place, y, w = case(tq, 12, 4, 6, 64, "float32")
    dO = torch.randn(12, 64, generator=g, device="cuda")
    dY, dw = tq.expert_combine_grad(dO, y, place, w)
    h = 2.0 ** -3                                  # linear: any step is exact but for rounding

    def f(y, w):
        return (tq.expert_combine(y, place, w).double() * dO.double()).sum()

    for t, j in ((0, 0), (5, 3), (11, 1)):
        e = torch.zeros_like(w)
        e[t, j] = h
        assert abs(float((f(y, w + e) - f(y, w - e)) / (2 * h)) - float(dw[t, j])) <= 2e-4
    for r, c in ((0, 0), (7, 63)):
        e = torch.zeros_like(y)
        e[r, c] = h
        got = float(dY[r, c]) if (place == r).any() else 0.0
        assert abs(float((f(y + e, w) - f(y - e, w)) / (2 * h)) - got) <= 2e-4


def test_combine_places_out_of_range_are_reported(tq):
    import torch
    y = torch.randn(4, 16, device="cuda")
    place = torch.tensor([[0, 4], [-2, 1], [-1, -1]], dtype=torch.int32, device="cuda")
    O = tq.expert_combine(y, place)
    assert tq.device_status() == 11
    assert torch.equal(O, torch.stack([y[0], y[1], torch.zeros_like(y[0])]))
    dY = torch.full((4, 16), 3.0, device="cuda")
    dO = torch.randn(3, 16, device="cuda")
    _, dw = tq.expert_combine_grad(dO, y, place, dY=dY)
    assert tq.device_status() == 11
    assert torch.equal(dY[:2], dO[:2]) and (dY[2:] == 3.0).all()
    assert dw[0, 1] == 0 and dw[1, 0] == 0 and (dw[2] == 0).all()


def test_gather_is_the_gradient_of_the_sum(tq):
    """With weights of one, the sum's gradient is the gather by the sort's tokens."""
    import torch
    g, token, place, y, _ = case(tq, 40, 4, 8, 128, "float32")
    dO = torch.randn(40, 128, generator=g, device="cuda")
    dY, _ = tq.expert_combine_grad(dO, y, place)
    assert torch.equal(dY, tq.expert_gather(dO, token))


# ------------------------------------------------------------------- together

@pytest.mark.parametrize("T,E,top,width,hidden", [(1, 8, 2, 256, 128), (16, 64, 8, 512, 256), (300, 12, 3, 272, 144),
                                                  (700, 8, 2, 512, 384)])
def test_layer(tq, T, E, top, width, hidden):
    """Router, sort, gathered operand, product, SwiGLU operand, product, sum: against
    64 bits, each step from the library's own input to it."""
    import torch
    g = gen(T)
    x = torch.randn(T, width, generator=g, device="cuda").bfloat16()
    router = torch.randn(E, width, generator=g, device="cuda").bfloat16()
    up = (torch.randn(E, 2 * hidden, width, generator=g, device="cuda") * width ** -0.5).bfloat16()
    down = (torch.randn(E, width, hidden, generator=g, device="cuda") * hidden ** -0.5).bfloat16()
    uq, us = tq.quantize_weights_f8(up)
    dq, ds = tq.quantize_weights_f8(down)
    rq, rs = tq.quantize_weights_f8(router)
    ws = tq.f8_workspace()
    lo = tq.linear_f8(*tq.quant_act_f8(x), rq, rs, ws, out="f32")
    ids, w = tq.expert_topk(lo, top)
    off, token, place = tq.expert_sort(ids, E)
    q, sx = tq.quant_act_f8(x, rows=token)
    gu = tq.linear_f8_experts(q, sx, off, uq, us, ws)
    hq, hs = tq.swiglu_quant_act_f8(gu[:, :hidden], gu[:, hidden:])
    y = tq.linear_f8_experts(hq, hs, off, dq, ds, ws)
    out = tq.expert_combine(y, place, w)
    assert tq.device_status() == 0
    want = torch.zeros(T, width, dtype=torch.float64, device="cuda")
    for t in range(T):
        for j in range(top):
            e = int(ids[t, j])
            v = x[t].double() @ up[e].double().t()
            h = ref.silu_mul(v[:hidden], v[hidden:])
            want[t] += float(w[t, j]) * (down[e].double() @ h)
    # e4m3's 2^-4 a value, on the operands of two products in a row
    err = float((out.double() - want).norm() / want.norm())
    assert err <= 0.1, err
