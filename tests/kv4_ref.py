"""A plain 64-bit model of the 4-bit cache, rotary positions and attention for
the tests, in numpy, written from the format and the formulas alone."""
import numpy as np

# angles in extended precision: a position of 2^31 needs more than fp64's 53 bits
TWO_PI = 2 * np.longdouble("3.14159265358979323846264338327950288")


def hadamard(n):
    h = np.ones((1, 1))
    while h.shape[0] < n:
        h = np.block([[h, h], [h, -h]])
    return h / np.sqrt(n)


def block_bytes(dim):
    return 16 * dim + 128


def nibbles(b):
    """Codes of a byte array, low nibble first, as signed numbers."""
    out = np.empty(b.shape[:-1] + (2 * b.shape[-1],), dtype=np.int64)
    out[..., 0::2] = (b & 15).astype(np.int64) - 8
    out[..., 1::2] = (b >> 4).astype(np.int64) - 8
    return out


def unpack(blocks, dim):
    """Blocks [..., bytes] -> (key codes, value codes [..., 16, dim], key
    scales, value scales [..., 16])."""
    lead = blocks.shape[:-1]
    k = nibbles(blocks[..., :8 * dim].reshape(lead + (16, dim // 2)))
    vb = blocks[..., 8 * dim:16 * dim].reshape(lead + (8, dim // 4, 2, 2))
    vb = np.swapaxes(vb, -3, -2).reshape(lead + (16, dim // 2))
    s = np.ascontiguousarray(blocks[..., 16 * dim:]).view(np.float32).astype(np.float64)
    return k, nibbles(vb), s[..., :16], s[..., 16:]


def pack(k, v, sk, sv):
    """The converse of unpack, for codes [..., 16, dim] and scales [..., 16]."""
    lead, dim = k.shape[:-2], k.shape[-1]
    out = np.zeros(lead + (block_bytes(dim),), dtype=np.uint8)

    def byte(c):
        u = (c + 8).astype(np.uint8)
        return u[..., 0::2] | (u[..., 1::2] << 4)
    out[..., :8 * dim] = byte(k).reshape(lead + (8 * dim,))
    b = byte(v).reshape(lead + (8, 2, dim // 4, 2))
    out[..., 8 * dim:16 * dim] = np.swapaxes(b, -3, -2).reshape(lead + (8 * dim,))
    s = np.concatenate([sk, sv], -1).astype(np.float32)
    out[..., 16 * dim:] = np.ascontiguousarray(s).view(np.uint8)
    return out


def quantise(x, dim):
    """(codes, scales, v / s before rounding) of rows x [..., dim]."""
    v = x @ hadamard(dim)
    s = (np.abs(v).max(-1) / 7.0).astype(np.float32).astype(np.float64)
    t = v / np.where(s > 0, s, 1.0)[..., None]
    return np.clip(np.rint(t), -7, 7).astype(np.int64), s, t


def pool_blocks(pool, npages, heads, dim, page):
    return pool.reshape(npages, heads, page // 16, block_bytes(dim))


def sequence(pool, table_row, length, page):
    """(K', V', key scales, value scales) of a sequence, rotated basis, fp64
    [heads, length, dim]; pool [pages, heads, blocks, bytes]."""
    heads, dim = pool.shape[1], (pool.shape[3] - 128) // 16
    n = -(-length // page)
    x = pool[np.asarray(table_row[:n], dtype=np.int64)]              # pages, heads, blocks, bytes
    k, v, sk, sv = unpack(x, dim)
    perm = lambda a: np.moveaxis(a, 1, 0).reshape((heads, n * page) + a.shape[4:])[:, :length]  # noqa: E731
    k, v, sk, sv = perm(k), perm(v), perm(sk), perm(sv)
    return k * sk[..., None], v * sv[..., None], sk, sv


def attend(q, kc, vc, length, new, scale, causal, window, widened=False):
    """o, lse, bound on |o - kernel's| before the bf16 rounding, and on lse's:
    q [new, hq, dim] fp64, kc / vc [heads, length, dim] of the rotated basis.

    Bounds: the kernel rounds each rotated query value to fp16, 2^-11 of it
    (its fp32 sums and exponential are far below that; twice it covers them):
    a score moves by at most eps = 2^-10 scale sum |q'||k'|, a weight by a
    factor e^(+-2 eps) after its normalisation; a weight times a value scale is
    rounded to fp16, 2^-11 of it (2^-10 with the sums').  Turned back, a row's
    error is at most the mean of its rotated ones times sqrt(dim).

    widened (more than 32 query rows a key/value head): keys and values are
    rounded too, a token's scale over its block's and its product with the code,
    2^-11 each, so three roundings where one was: 2^-9 covers them.  A weight
    over its value's scale below the row's largest by 2^14 loses bits, 2^-25 of
    that largest one's (2^-22 with the scale's margin of 4 and code's of 8), and
    a scale 2^28 below its block's largest 2^-39 of that one's."""
    n, hq, dim = q.shape
    heads = kc.shape[0]
    g = hq // heads
    H = hadamard(dim)
    o = np.zeros((n, hq, dim))
    lse = np.full((n, hq), -np.inf)
    eo = np.zeros((n, hq))
    el = np.zeros((n, hq))
    for i in range(n):
        p = length - new + i
        hi = 0 if p < 0 else (min(length, p + 1) if causal else length)
        lo = max(0, p - window + 1) if window else 0
        if hi <= lo:
            continue
        for h in range(hq):
            qr = q[i, h] @ H
            k, v = kc[h // g, lo:hi], vc[h // g, lo:hi]
            x = scale * (k @ qr)
            m = x.max()
            w = np.exp(x - m)
            tot = w.sum()
            w /= tot
            o[i, h] = (w @ v) @ H
            lse[i, h] = m + np.log(tot)
            eps = 2.0 ** (-9 if widened else -10) * scale * (np.abs(k) @ np.abs(qr)).max()
            el[i, h] = eps + 2.0 ** -20 * (1 + abs(lse[i, h]))
            eo[i, h] = (np.expm1(2 * eps) + 2.0 ** (-9 if widened else -10)) * (w @ np.abs(v)).sum() / np.sqrt(dim)
            if widened:
                eo[i, h] += (hi - lo) * 2.0 ** -22 * w.max() * np.abs(v).max() * np.sqrt(dim)
    return o, lse, eo, el


def rope(x, pos, inv_freq, axis, interleaved):
    """x [tokens, heads, dim] fp64, pos [axes, tokens]."""
    y = x.copy()
    pairs = len(inv_freq)
    for p in range(pairs):
        a, b = (2 * p, 2 * p + 1) if interleaved else (p, p + pairs)
        t = np.remainder(pos[axis[p]].astype(np.longdouble) * np.longdouble(inv_freq[p]), TWO_PI)
        c, s = np.cos(t).astype(np.float64)[:, None], np.sin(t).astype(np.float64)[:, None]
        y[:, :, a] = x[:, :, a] * c - x[:, :, b] * s
        y[:, :, b] = x[:, :, b] * c + x[:, :, a] * s
    return y
