"""The root-mean-square norm with its residual's addition, into the rotated
8-bit operand (rows and tiled) and into bf16, against 64 bits.

Bars, set before the first run:
  - h equals bf16(x + r) formed in fp32, bit for bit;
  - y within half a bf16 step of the 64-bit value plus 2^-20 of it (the sum of
    squares of at most 2^14 values in fp32 pairs and trees, the reciprocal
    root and two products: each below 2^-22);
  - token scales within 2^-18 of the 64-bit ones (the same, and the butterfly's
    eight sums); codes equal but for at most 0.1%, there by one;
  - the tiled operand's codes and scales equal the rows', bit for bit.
"""
import numpy as np
import pytest

import kv4_ref as ref
from helpers import REL_L2_Y, act_trailer, check_codes_close, rel_l2, to_np, untile_codes

pytestmark = pytest.mark.gpu


def inputs(M, K, seed, pad=0):
    import torch
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(M, K + pad))
    x[:, rng.integers(0, K + pad, max(1, K // 400))] *= 40.0
    gamma = 1.0 + 0.2 * rng.normal(size=K)
    return torch.from_numpy(x).cuda().bfloat16(), torch.from_numpy(gamma).cuda().float()


def exact(h, gamma, eps):
    h = h.double().cpu().numpy()
    ms = (h * h).mean(1, keepdims=True) + np.float64(np.float32(eps))
    y = h * np.where(ms > 0, 1 / np.sqrt(np.where(ms > 0, ms, 1)), 0) * gamma.double().cpu().numpy()
    K = y.shape[1]
    v = np.concatenate([y[:, g:g + 256] @ ref.hadamard(min(256, K - g)) for g in range(0, K, 256)], 1)
    s = np.abs(v).max(1) / 127.0
    q = np.clip(np.rint(v / np.where(s > 0, s, 1)[:, None]), -127, 127).astype(np.int64)
    return y, q, s


def check(x, gamma, eps, h, Xq, sx, Y=None):
    y, q, s = exact(h, gamma, eps)
    if Y is not None:
        got = Y.double().cpu().numpy()
        assert np.all(np.abs(got - y) <= np.abs(y) * (2.0 ** -8 + 2.0 ** -20))
    if sx is not None:
        assert np.all(np.abs(to_np(sx).astype(np.float64) - s) <= 2.0 ** -18 * s)
        check_codes_close(to_np(Xq), q)


SHAPES = [(1, 32), (1, 896), (3, 64), (2, 128), (130, 4096), (64, 768 + 32), (5, 256), (33, 1024 + 64), (3, 16384),
          (2, 16384 - 128), (9, 4096 + 128), (700, 512)]


@pytest.mark.parametrize("M,K", SHAPES)
@pytest.mark.parametrize("residual", [False, True])
def test_norm_rows_and_tiled(tq, M, K, residual):
    import torch
    x, gamma = inputs(M, K, K + M)
    r = inputs(M, K, K + M + 1)[0] if residual else None
    H = torch.empty_like(x)
    Y = torch.empty_like(x)
    Xq, sx = tq.rmsnorm_quant_act(x, gamma, 1e-6, R=r, H=H, Y=Y)
    h = (x.float() + r.float()).bfloat16() if residual else x
    assert torch.equal(H, h)
    check(x, gamma, 1e-6, h, Xq, sx, Y)
    assert torch.equal(tq.rmsnorm(x, gamma, 1e-6, R=r), Y)
    H2 = torch.empty_like(x)
    At, st = tq.rmsnorm_quant_act_tiled(x, gamma, 1e-6, R=r, H=H2)
    assert torch.equal(st, sx) and torch.equal(H2, h)
    assert np.array_equal(untile_codes(At, M, K), to_np(Xq))
    tr = act_trailer(tq, At, M, K)
    c = to_np(Xq).astype(np.int64)
    assert tr[0] == np.abs(c).sum(1).max() and tr[6] == (c * c).sum(1).max()
    a, b = tq.rmsnorm_quant_act(x, gamma, 1e-6, R=r)        # no H, no Y; the same bytes again
    assert torch.equal(a, Xq) and torch.equal(b, sx)
    assert tq.device_status() == 0


@pytest.mark.parametrize("place", ["X", "R"])
def test_residual_stream_in_place_strided(tq, place):
    import torch
    M, K = 41, 2048 + 64
    bx, gamma = inputs(M, K, 1, pad=72)
    br, _ = inputs(M, K, 2, pad=72)
    x, r = bx[:, 8:8 + K], br[:, 16:16 + K]
    kx, kr = bx.clone(), br.clone()
    h = (x.float() + r.float()).bfloat16()
    dst = x if place == "X" else r
    yb = torch.full((M, K + 24), 5.0, dtype=torch.bfloat16, device="cuda")
    Xq, sx = tq.rmsnorm_quant_act(x, gamma, 1e-5, R=r, H=dst, Y=yb[:, :K])
    assert torch.equal(dst, h) and bool((yb[:, K:] == 5.0).all())
    check(x, gamma, 1e-5, h, Xq, sx, yb[:, :K])
    same, other, at = (bx, br, 8) if place == "X" else (br, bx, 16)
    k_same, k_other = (kx, kr) if place == "X" else (kr, kx)
    assert torch.equal(other, k_other)
    assert torch.equal(same[:, :at], k_same[:, :at]) and torch.equal(same[:, at + K:], k_same[:, at + K:])


def test_special_rows(tq):
    """Rows of zeros (with eps = 0 too), of one value, of one outlier, and
    rows that cancel their residual."""
    import torch
    M, K = 6, 896
    x, gamma = inputs(M, K, 3)
    x[0] = 0
    x[1] = 1.375
    x[2] = 0
    x[2, 777] = -3.0
    r = torch.zeros_like(x)
    r[3] = -x[3]
    r[4] = x[4] * 256
    for eps in (0.0, 1e-6):
        H, Y = torch.empty_like(x), torch.empty_like(x)
        Xq, sx = tq.rmsnorm_quant_act(x, gamma, eps, R=r, H=H, Y=Y)
        check(x, gamma, eps, H, Xq, sx, Y)
        for m in (0, 3):
            assert not Xq[m].any() and not Y[m].any() and float(sx[m]) == 0.0


def test_norm_feeds_the_products(tq):
    """The norm's operands through the A8 products (rows and tiled weights):
    exact sums of the same codes, and through the A16 product."""
    import torch
    M, N, K = 20, 300, 896
    x, gamma = inputs(M, K, 4)
    W = inputs(N, K, 5)[0] * 0.02
    codes, sw = tq.quantize_weights(W, 8)
    Xq, sx = tq.rmsnorm_quant_act(x, gamma)
    At, st = tq.rmsnorm_quant_act_tiled(x, gamma)
    acc = to_np(tq.linear_q8(Xq, sx, codes, sw, N, 8, out="i32"))
    assert np.array_equal(acc, to_np(Xq).astype(np.int64) @ to_np(codes).astype(np.int64).T)
    Wt = tq.tile_weights(codes, N, K, 8)
    assert np.array_equal(to_np(tq.linear_tt(At, st, M, K, Wt, sw, N, 8, out="i32")), acc)
    y = tq.rmsnorm(x, gamma)
    a16 = tq.linear(y, codes, sw, N, 8, "W8A16")
    v = np.concatenate([y.double().cpu().numpy()[:, g:g + 256] @ ref.hadamard(min(256, K - g))
                        for g in range(0, K, 256)], 1)
    vb = torch.from_numpy(v).bfloat16().double().numpy()
    want = (vb @ to_np(codes).astype(np.float64).T) * to_np(sw)
    assert rel_l2(to_np(a16), want) <= 100 * REL_L2_Y       # bf16 ties of x' may round the other way
    assert tq.device_status() == 0


@pytest.mark.parametrize("K", [64, 896, 4096 + 128])
def test_rows_that_are_not_finite(tq, K):
    """A NaN anywhere in a row, or infinities that meet in the residual's
    addition, make all of the row NaN in bf16; the other rows are as without."""
    import torch
    M = 7
    x, gamma = inputs(M, K, K)
    r = inputs(M, K, K + 1)[0]
    want = tq.rmsnorm(x, gamma, R=r)
    x[1, K - 1] = float("nan")
    x[3, 0] = float("inf")
    r[3, 0] = -float("inf")
    r[5, K // 2] = float("nan")
    got = tq.rmsnorm(x, gamma, R=r)
    odd = [1, 3, 5]
    assert got[odd].isnan().all()
    keep = [0, 2, 4, 6]
    assert torch.equal(got[keep], want[keep]) and got[keep].isfinite().all()
    assert tq.rmsnorm(x, gamma)[1].isnan().all()
    assert tq.device_status() == 0
