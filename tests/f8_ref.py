"""Plain 64-bit forms of the 8-bit floating-point products and of a layer's experts,
from the formulas alone (torch, any device)."""
import math

import torch

BLOCK, MOST = 128, 448.0


def decode(codes):
    """e4m3 bytes as 64-bit values: sign, four bits of exponent (bias 7), three of
    mantissa; 0x7F and 0xFF are NaN."""
    c = codes.to(torch.int64)
    e, m = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e > 0, (8 + m) * torch.exp2((e - 10).double()), m * 2.0 ** -9)
    v = torch.where((c & 127) == 127, math.nan, v)
    return torch.where(c >= 128, -v, v)


def encode(v):
    """The nearest e4m3 byte of 64-bit values within +-448, ties to the even code."""
    table = decode(torch.arange(127, device=v.device))            # 0 .. 448, rising
    a = v.abs()
    hi = torch.searchsorted(table, a).clamp(1, 126)
    lo = hi - 1
    dl, dh = a - table[lo], table[hi] - a
    c = torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return torch.where(torch.signbit(v), c + 128, c).to(torch.uint8)


def power_scale(amax):
    """The smallest power of two 2^j, j >= -126, with amax / 2^j <= 448 (a Python
    number: searched for, not computed by a logarithm)."""
    if amax == 0:
        return 0.0
    if not math.isfinite(amax):
        return math.nan
    j = -126
    while amax > MOST * 2.0 ** j:
        j += 1
    return 2.0 ** j


def quantise(x, rows=1):
    """(codes, scales [blocks of rows, blocks of columns]) of 64-bit x by blocks of
    `rows` rows and 128 columns."""
    m, k = x.shape
    codes = torch.zeros(m, k, dtype=torch.uint8, device=x.device)
    scales = torch.zeros(-(-m // rows), -(-k // BLOCK), dtype=torch.float64, device=x.device)
    for i in range(scales.shape[0]):
        for j in range(scales.shape[1]):
            at = slice(i * rows, (i + 1) * rows), slice(j * BLOCK, (j + 1) * BLOCK)
            b = x[at]
            s = power_scale(float("nan") if not torch.isfinite(b).all() else float(b.abs().max()))
            scales[i, j] = s
            if s > 0:
                codes[at] = encode(b / s)
    return codes, scales


def values(codes, scales, rows=1):
    """What codes and their blocks' scales stand for."""
    m, k = codes.shape
    s = scales.double().repeat_interleave(rows, 0)[:m].repeat_interleave(BLOCK, 1)[:, :k]
    return decode(codes) * s


def product(xq, sx, wq, sw):
    """(Y, the sum of the terms' magnitudes), both 64-bit: sx as the library has it,
    [blocks, M]."""
    x, w = values(xq, sx.t()), values(wq, sw, BLOCK)
    return x @ w.t(), x.abs() @ w.abs().t()


def product_bar(K, S, Y, bf16):
    """How far a product may be off.  Each of a block's 128 additions rounds or cuts
    off at most 2^-23 of what cannot pass the sum S of all magnitudes (2^-16 in all);
    the scales' product, the fma of each block and the joining of up to eight parts
    round by 2^-24 each; a bf16 result by half a step, 2^-8 of it."""
    bar = S * (2.0 ** -16 + (-(-K // BLOCK) + 10) * 2.0 ** -24)
    return bar + (Y.abs() * 2.0 ** -8 if bf16 else 0.0) * (1 + 2.0 ** -8)


def silu_mul(g, u):
    return g * torch.sigmoid(g) * u


def topk(x, top):
    """ids by sorting pairs (value down, index up) in Python; -inf is never chosen, a
    NaN comes first."""
    ids = torch.full((x.shape[0], top), -1, dtype=torch.int32)
    for t, row in enumerate(x.double().cpu().tolist()):
        order = sorted((i for i, v in enumerate(row) if v != -math.inf),
                       key=lambda i: (0 if math.isnan(row[i]) else 1, -row[i], i))
        for j, i in enumerate(order[:top]):
            ids[t, j] = i
    return ids


def weights(x, ids, renorm):
    """Softmax weights of the choices, 64-bit on x's device."""
    x, ids = x.double(), ids.to(x.device).long()
    m = x.max(1, keepdim=True).values
    p = torch.exp(x - torch.where(torch.isfinite(m), m, 0.0))
    w = torch.where(ids >= 0, torch.gather(p, 1, ids.clamp(min=0)), 0.0)
    total = w.sum(1, keepdim=True) if renorm else p.sum(1, keepdim=True)
    return w / torch.where(total > 0, total, 1.0)


def sort(ids, experts):
    """(offsets, token, place) by walking the choices."""
    T, top = ids.shape
    flat = ids.reshape(-1).tolist()
    offsets, token, place = [0], [], [-1] * len(flat)
    for e in range(experts):
        for f, i in enumerate(flat):
            if i == e:
                place[f] = len(token)
                token.append(f // top)
        offsets.append(len(token))
    token += [-1] * (len(flat) - len(token))
    i32 = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    return i32(offsets), i32(token), i32(place).view(T, top)
