"""Rotary positions with one or more axes against 64 bits.

Bar, set before the first run: half a bf16 step of the 64-bit value (2^-8 of
it) plus 2^-20 of |x0| + |x1| (the reduced angle rounded to fp32, 2^-23 of at
most pi; sine and cosine within two units of 2^-24; two products and a sum).
"""
import numpy as np
import pytest

import kv4_ref as ref

pytestmark = pytest.mark.gpu


def f64(t):
    return t.double().cpu().numpy()


def make(tokens, heads, dim, pairs, axes, span, seed, lo=0):
    import torch
    rng = np.random.default_rng(seed)
    x = torch.from_numpy(rng.normal(size=(tokens, heads, dim))).cuda().bfloat16()
    pos = rng.integers(lo, span, size=(axes, tokens)).astype(np.int32)
    freq = (10000.0 ** (-np.arange(pairs) / pairs)).astype(np.float32)
    axis = rng.integers(0, axes, pairs)
    return x, pos, freq, axis


def check(x, y, pos, freq, axis, inter):
    want = ref.rope(f64(x), pos, freq, axis, inter)
    p = len(freq)
    xa = np.abs(f64(x))
    size = np.zeros_like(xa)
    a, b = (np.arange(0, 2 * p, 2), np.arange(1, 2 * p, 2)) if inter else (np.arange(p), np.arange(p, 2 * p))
    size[..., a] = size[..., b] = xa[..., a] + xa[..., b]
    assert np.all(np.abs(f64(y) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * size)
    assert np.array_equal(f64(y)[..., 2 * p:], f64(x)[..., 2 * p:])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,heads,dim,pairs,axes", [
    (1, 1, 64, 32, 1), (7, 40, 128, 64, 1), (300, 3, 128, 64, 3), (33, 5, 256, 64, 2), (65, 2, 64, 13, 4),
    (19, 7, 8, 4, 1), (5, 3, 72, 36, 3), (2, 2, 128, 1, 1), (11, 6, 80, 20, 2), (4, 130, 128, 60, 3)])
def test_rope(tq, interleaved, tokens, heads, dim, pairs, axes):
    import torch
    x, pos, freq, axis = make(tokens, heads, dim, pairs, axes, 5000, tokens + dim)
    spec = tq.RopeSpec(torch.from_numpy(freq).cuda(), axis.tolist(), interleaved)
    y = tq.rope(x, torch.from_numpy(pos).cuda(), spec)
    check(x, y, pos, freq, axis, interleaved)
    z = x.clone()
    assert tq.rope(z, torch.from_numpy(pos).cuda(), spec, Y=z) is z and torch.equal(z, y)
    assert tq.device_status() == 0


@pytest.mark.parametrize("interleaved", [False, True])
def test_extreme_positions(tq, interleaved):
    """The last int32 positions and negative ones turn as exactly as the first
    (the model's angle needs more than 53 bits: extended precision)."""
    import torch
    x, _, freq, axis = make(8, 2, 128, 64, 1, 10, 3)
    pos = np.array([[2 ** 31 - 1, -2 ** 31, 2 ** 30 + 1, -1, 0, 1, 131071, -12345]], dtype=np.int32)
    spec = tq.RopeSpec(torch.from_numpy(freq).cuda(), None, interleaved)
    y = tq.rope(x, torch.from_numpy(pos).cuda(), spec)
    check(x, y, pos, freq, np.zeros(64, int), interleaved)


@pytest.mark.parametrize("interleaved", [False, True])
def test_strided_rows_leave_the_rest_alone(tq, interleaved):
    """Query and key heads of a fused projection's row in place, the value
    heads beside them untouched; positions with a stride between the axes."""
    import torch
    x, pos, freq, axis = make(50, 12, 128, 64, 3, 90, 4)
    keep = x.clone()
    big = torch.zeros(3, 64, dtype=torch.int32, device="cuda")
    big[:, :50] = torch.from_numpy(pos).cuda()
    spec = tq.RopeSpec(torch.from_numpy(freq).cuda(), axis.tolist(), interleaved)
    q = x[:, :9]
    tq.rope(q, big[:, :50], spec, Y=q)
    check(keep[:, :9], q, pos, freq, axis, interleaved)
    assert torch.equal(x[:, 9:], keep[:, 9:])


def test_positions_in_scores_are_relative(tq):
    """A query's product with a key depends on their distance alone."""
    import torch
    x, _, freq, _ = make(1, 2, 128, 64, 1, 10, 5)
    spec = tq.RopeSpec(torch.from_numpy(freq).cuda())
    def at(p):
        return f64(tq.rope(x, torch.tensor([[p]], dtype=torch.int32, device="cuda"), spec))[0]
    near = at(3)[0] @ at(10)[1]
    far = at(100003)[0] @ at(100010)[1]
    norm = np.linalg.norm(f64(x)[0, 0]) * np.linalg.norm(f64(x)[0, 1])
    assert abs(near - far) <= 4 * 2.0 ** -8 * norm / np.sqrt(128) * 4     # four roundings of 128 values at random
