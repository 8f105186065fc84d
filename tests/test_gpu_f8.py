"""e4m3 operands and their products against 64 bits.

Bars, set before the first run:
  - codes and scales equal the 64-bit ones bit for bit (x / s is exact, so there is
    one rounding on both sides); for the SwiGLU, formed in fp32 with approximate
    exponential and division, codes are those of a value within 2^-19 of the exact
    one: they differ on at most 1 % and there by one code, and a block's scale may
    be the neighbouring power only where its largest value is within 2^-19 of the
    border;
  - products: f8_ref.product_bar.
"""
import numpy as np
import pytest

import f8_ref as ref

pytestmark = pytest.mark.gpu


def gen(seed):
    import torch
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape):
    import torch
    return torch.randn(*shape, generator=g, device="cuda")


def rows(g, m, k, pad=0):
    """bf16 rows with outliers, some tiny values and a block of zeros, strided."""
    import torch
    x = normal(g, m, k + pad)
    x[:, torch.randint(0, k, (max(1, k // 300),), generator=g, device="cuda")] *= 40.0
    x[:, ::7] *= 2.0 ** -12
    x = x.bfloat16()
    if k > 128:
        x[m // 2, :128] = 0.0
    return x[:, :k]


SIZES = [(1, 16), (1, 128), (3, 144), (2, 896), (64, 2000), (130, 4096), (5, 512 + 16), (9, 65536)]


@pytest.mark.parametrize("M,K", SIZES)
def test_rows(tq, M, K):
    import torch
    x = rows(gen(M + K), M, K, 8 * (M % 3))
    q, s = tq.quant_act_f8(x)
    wq, ws = ref.quantise(x.double().cpu()) if M * K < 200000 else (None, None)
    if wq is None:        # every seventh row is enough of a large one
        pick = list(range(0, M, 7))
        wq, ws = ref.quantise(x[pick].double().cpu())
        q, s = q[pick], s[:, pick]
    assert torch.equal(q.cpu(), wq)
    assert torch.equal(s.cpu().double(), ws.t())
    assert tq.device_status() == 0


def test_rows_borders(tq):
    """Largest values on both sides of 448 * 2^j, ties, the smallest and largest bf16."""
    import torch
    x = torch.zeros(12, 256)
    for i, top in enumerate((448.0, 450.0, 1.75, 1.7578125, 2.0 ** -133, 2.0 ** -118, 3.3895e38, 2.0 ** -126, 0.0,
                             1.0, 447.0, 2.0 ** -120)):
        x[i, 3] = -top
        x[i, 4:60] = torch.linspace(-1, 1, 56) * top
        x[i, 128:256] = top * 2.0 ** -torch.arange(128.0)
    x = x.bfloat16().cuda()
    q, s = tq.quant_act_f8(x)
    wq, ws = ref.quantise(x.double().cpu())
    assert torch.equal(s.cpu().double(), ws.t())
    assert torch.equal(q.cpu(), wq)


def test_rows_not_finite(tq):
    import torch
    x = torch.ones(3, 256).bfloat16().cuda()
    x[0, 5], x[1, 200], x[2, 0] = float("nan"), float("inf"), float("-inf")
    q, s = tq.quant_act_f8(x)
    nan = torch.isnan(s).cpu().tolist()
    assert nan == [[True, False, True], [False, True, False]]
    assert (q[0, :128] == 0).all() and (q[1, 128:] == 0).all() and (q[1, :128] == q[1, 0]).all()


@pytest.mark.parametrize("M,K", [(1, 16), (40, 896), (7, 2000)])
def test_rows_gathered(tq, M, K):
    import torch
    g = gen(K)
    x = rows(g, 19, K, 16)
    pick = torch.randint(-1, 19, (M,), generator=g, device="cuda", dtype=torch.int32)
    q = torch.full((M, K), 77, dtype=torch.uint8, device="cuda")
    s = torch.full((-(-K // 128), M), 5.0, device="cuda")
    tq.quant_act_f8(x, rows=pick, Xq=q, sx=s)
    fq, fs = tq.quant_act_f8(x)
    for m, r in enumerate(pick.tolist()):
        assert torch.equal(q[m], fq[r] if r >= 0 else torch.full_like(q[m], 77))
        assert torch.equal(s[:, m], fs[:, r] if r >= 0 else torch.full_like(s[:, m], 5.0))
    assert tq.device_status() == 0


def test_rows_out_of_range_are_reported(tq):
    import torch
    x = torch.ones(4, 128).bfloat16().cuda()
    q = torch.full((5, 128), 77, dtype=torch.uint8, device="cuda")
    s = torch.full((1, 5), 5.0, device="cuda")
    tq.quant_act_f8(x, rows=torch.tensor([0, 4, -2, 3, -1], dtype=torch.int32, device="cuda"), Xq=q, sx=s)
    assert tq.device_status() == 11
    assert (q[[1, 2, 4]] == 77).all() and s[0].tolist() == [2.0 ** -8, 5.0, 5.0, 2.0 ** -8, 5.0]
    assert tq.device_status() == 0


@pytest.mark.parametrize("M,K,fused", [(1, 16, False), (33, 1024, True), (6, 2000, True)])
def test_swiglu_rows(tq, M, K, fused):
    import torch
    g = gen(M)
    both = (3.0 * normal(g, M, 2 * K)).bfloat16()
    G, U = (both[:, :K], both[:, K:]) if fused else (both[:, :K].contiguous(), both[:, K:].contiguous())
    q, s = tq.swiglu_quant_act_f8(G, U)
    h = ref.silu_mul(G.double(), U.double()).cpu()
    wq, ws = ref.quantise(h)
    s = s.cpu().double().t()
    near = (h.abs() * 2.0 ** -19).nan_to_num()
    for i, j in zip(*np.nonzero((s != ws).numpy())):
        a = float(h[i, 128 * j:128 * j + 128].abs().max())
        assert abs(a / (448.0 * min(s[i, j], ws[i, j])) - 1.0) <= 2.0 ** -19
    same = (s == ws).repeat_interleave(128, 1)[:, :K]
    d = (ref.decode(q.cpu()) - ref.decode(wq)).abs()
    step = torch.maximum(ref.decode(wq).abs() * 2.0 ** -3, torch.tensor(2.0 ** -9).double())
    assert (d[same] <= step[same]).all()
    assert int((d[same] > 0).sum()) <= 0.01 * d.numel()
    assert near.shape == d.shape


@pytest.mark.parametrize("N,K", [(1, 16), (128, 128), (129, 144), (300, 896), (64, 2000)])
def test_weights(tq, N, K):
    import torch
    W = rows(gen(N), N, K, 8)
    q, s = tq.quantize_weights_f8(W)
    wq, ws = ref.quantise(W.double().cpu(), 128)
    assert torch.equal(q.cpu(), wq) and torch.equal(s.cpu().double(), ws)


def test_weights_of_experts(tq):
    import torch
    W = torch.stack([rows(gen(i), 130, 272).contiguous() for i in range(3)])
    q, s = tq.quantize_weights_f8(W)
    for e in range(3):
        a, b = tq.quantize_weights_f8(W[e])
        assert torch.equal(q[e], a) and torch.equal(s[e], b)


# ------------------------------------------------------------------ the products

def matrix(g, *shape):
    """Published weights: e4m3 codes of every kind but NaN, scales that are no powers."""
    import torch
    *lead, n, k = shape
    codes = torch.randint(0, 256, shape, generator=g, device="cuda", dtype=torch.int32).to(torch.uint8)
    codes = torch.where((codes & 127) == 127, codes - 1, codes)
    small = torch.rand(shape, generator=g, device="cuda") < 0.9      # most of them not huge
    codes = torch.where(small, (codes & 0x87) | (((codes >> 3) & 7) << 3), codes)
    scales = torch.rand(*lead, -(-n // 128), -(-k // 128), generator=g, device="cuda") * 0.01 + 0.001
    return codes.contiguous(), scales


def framed(M, N, dtype, pad):
    """(whole, the [M, N] part) of a buffer filled with a mark."""
    import torch
    whole = torch.full((M + 2, N + pad), 3.0, dtype=dtype, device="cuda")
    return whole, whole[1:M + 1, :N]


def check_frame(whole, M, N):
    assert (whole[0] == 3.0).all() and (whole[M + 1] == 3.0).all() and (whole[:, N:] == 3.0).all()


def check(Y, want, S, K):
    import torch
    err = (Y.double() - want).abs()
    bar = ref.product_bar(K, S, want, Y.dtype == torch.bfloat16)
    assert not torch.isnan(Y).any()
    assert (err <= bar).all(), f"off by {float((err / bar).max())} of the bar"


PRODUCTS = [(1, 1, 16), (1, 8, 128), (1, 4864, 896), (2, 127, 144), (3, 128, 16), (8, 129, 4864), (16, 896, 4864),
            (17, 300, 2000), (31, 4096, 4096), (32, 1, 4096), (33, 256, 112), (48, 12288, 512), (63, 300, 272), (64, 1100, 2000),
            (65, 513, 128), (96, 4864, 896), (128, 256, 8192), (129, 255, 1040), (200, 1000, 2000), (255, 384, 256),
            (256, 256, 128), (257, 257, 144), (300, 3, 4096), (513, 640, 1024), (1013, 1100, 2000),
            (1025, 2048, 2048), (4, 64, 65536), (600, 130, 16384)]


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_product(tq, M, N, K, out):
    import torch
    g = gen(M * 7 + N)
    q, sx = tq.quant_act_f8(rows(g, M, K))
    Wq, sw = matrix(g, N, K)
    ws = tq.f8_workspace()
    whole, Y = framed(M, N, torch.float32 if out == "f32" else torch.bfloat16, (0, 8, 5)[M % 3])
    tq.linear_f8(q, sx, Wq, sw, ws, out=out, Y=Y)
    want, S = ref.product(q, sx, Wq, sw)
    check(Y, want, S, K)
    check_frame(whole, M, N)
    again = tq.linear_f8(q, sx, Wq, sw, ws, out=out)
    assert torch.equal(again, Y)
    assert tq.device_status() == 0


# many tokens: tiles of 128 columns; one round, two, and a last one that is cut along K;
# columns that end inside a tile's half
@pytest.mark.parametrize("M,N,K", [(70, 12288, 256), (128, 12200, 400), (300, 4096, 640), (640, 4096, 12288),
                                   (777, 12288, 512), (700, 12298, 256)])
def test_product_forms(tq, M, N, K):
    test_product(tq, M, N, K, "bf16")


# rows of Y that begin anywhere: many tokens, columns that end inside a word
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("M,N", [(777, 6001), (778, 6002), (779, 6003), (902, 6004)])
def test_product_unaligned_rows(tq, M, N, out):
    test_product(tq, M, N, 272, out)


def test_product_of_weights_written_just_before(tq):
    """The weights' kernel and the product with nothing in between."""
    import torch
    g = gen(5)
    N, K = 4096, 2048
    a, b = (torch.randn(N, K, generator=g, device="cuda").bfloat16() for _ in range(2))
    for M in (4, 300):
        q, sx = tq.quant_act_f8(rows(g, M, K))
        ws = tq.f8_workspace()
        want = [tq.linear_f8(q, sx, *tq.quantize_weights_f8(w), ws, out="f32") for w in (a, b)]
        Wq, sw = tq.quantize_weights_f8(a)
        got = []
        for i in range(12):
            tq.quantize_weights_f8((a, b)[i % 2], Wq, sw)
            got.append(tq.linear_f8(q, sx, Wq, sw, ws, out="f32"))
        for i, y in enumerate(got):
            assert torch.equal(y, want[i % 2])


def test_product_empty(tq):
    import torch
    ws = tq.f8_workspace()
    q = torch.empty(0, 128, dtype=torch.uint8, device="cuda")
    sx = torch.empty(1, 0, device="cuda")
    Wq, sw = matrix(gen(0), 64, 128)
    assert tq.linear_f8(q, sx, Wq, sw, ws).shape == (0, 64)


@pytest.mark.parametrize("M", [4, 300])
def test_product_not_finite(tq, M):
    """A NaN scale, or a NaN code, reaches the outputs that meet it and no others."""
    import torch
    g = gen(5)
    N, K = 300, 512
    q, sx = tq.quant_act_f8(rows(g, M, K))
    Wq, sw = matrix(g, N, K)
    sx[1, 2] = float("nan")                 # row 2
    sw[1, 3] = float("nan")                 # columns 128 .. 255
    Wq[270, 17] = 0x7F                      # column 270
    Wq[271, 18] = 0xFF
    Y = tq.linear_f8(q, sx, Wq, sw, tq.f8_workspace(), out="f32")
    bad = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    bad[2], bad[:, 128:256], bad[:, 270:272] = True, True, True
    assert torch.equal(torch.isnan(Y), bad)
    want, S = ref.product(q, sx, Wq, sw)
    ok = ~bad
    assert ((Y.double() - want).abs()[ok] <= ref.product_bar(K, S, want, False)[ok]).all()


def test_product_scales_of_zero_and_large(tq):
    import torch
    g = gen(6)
    M, N, K = 70, 256, 384
    q, sx = tq.quant_act_f8(rows(g, M, K))
    Wq, sw = matrix(g, N, K)
    sx[0] = 0.0
    sx[1, :40] *= 2.0 ** 60
    sw[0, 1] *= 2.0 ** 40
    sw[1, 2] *= 2.0 ** -80
    Y = tq.linear_f8(q, sx, Wq, sw, tq.f8_workspace(), out="f32")
    want, S = ref.product(q, sx, Wq, sw)
    check(Y, want, S, K)


def offsets_of(counts, first=0):
    import torch
    return torch.tensor([first, *(first + np.cumsum(counts)).tolist()], dtype=torch.int32, device="cuda")


EXPERTS = [([3], 64, 128, 4), ([1, 0, 2, 1], 129, 144, 6), ([0, 0, 0], 64, 128, 5), ([16, 1, 0, 7, 33], 300, 272, 60),
           ([1] * 20 + [0] * 10, 896, 512, 25), ([40, 2, 70, 0, 5, 64], 256, 2000, 181),
           ([200, 1, 0, 513, 77, 300], 384, 512, 1200), ([0, 1000, 0], 130, 256, 1000),
           ([256, 512, 255, 257], 512, 1024, 1300), ([5, 90] * 16, 640, 384, 1520), ([2] * 1024, 16, 32, 2048),
           ([0] * 1023 + [9], 40, 144, 9), ([31, 33] * 4, 4096, 2048, 256)]


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("counts,N,K,M", EXPERTS)
def test_experts(tq, counts, N, K, M, out):
    import torch
    g = gen(len(counts) + N)
    first = min(1, M - sum(counts))
    off = offsets_of(counts, first)
    q, sx = tq.quant_act_f8(rows(g, M, K))
    Wq, sw = matrix(g, len(counts), N, K)
    ws = tq.f8_workspace()
    whole, Y = framed(M, N, torch.float32 if out == "f32" else torch.bfloat16, (8, 0, 3)[N % 3])
    tq.linear_f8_experts(q, sx, off, Wq, sw, ws, out=out, Y=Y)
    ends = off.tolist()
    for e, (a, b) in enumerate(zip(ends, ends[1:])):
        if a < b:
            want, S = ref.product(q[a:b], sx[:, a:b], Wq[e], sw[e])
            check(Y[a:b], want, S, K)
    check_frame(whole, M, N)
    assert (Y[:first] == 3.0).all() and (Y[ends[-1]:] == 3.0).all()      # rows that no expert has
    again = torch.full_like(Y, 3.0)
    tq.linear_f8_experts(q, sx, off, Wq, sw, ws, out=out, Y=again)
    assert torch.equal(again, Y)
    assert tq.device_status() == 0


@pytest.mark.parametrize("M", [40, 3000])
@pytest.mark.parametrize("bad", ["backwards", "negative", "past"])
def test_experts_bad_ranges_are_empty_and_reported(tq, bad, M):
    import torch
    g = gen(9)
    N, K = 256, 256
    q, sx = tq.quant_act_f8(rows(g, M, K))
    Wq, sw = matrix(g, 4, N, K)
    ends = {"backwards": [0, 20, 10, 30, 40], "negative": [-3, 20, 21, 30, 40], "past": [0, 20, 21, 30, M + 1]}[bad]
    Y = torch.full((M, N), 3.0, device="cuda")
    tq.linear_f8_experts(q, sx, torch.tensor(ends, dtype=torch.int32, device="cuda"), Wq, sw, tq.f8_workspace(),
                         out="f32", Y=Y)
    assert tq.device_status() == 11
    seen = torch.zeros(M, dtype=torch.bool)
    for e, (a, b) in enumerate(zip(ends, ends[1:])):
        if 0 <= a < b <= M and a >= max(ends[:e + 1]):     # no row is two experts'
            want, S = ref.product(q[a:b], sx[:, a:b], Wq[e], sw[e])
            check(Y[a:b], want, S, K)
            seen[a:b] = True
    assert (Y[~seen.cuda()] == 3.0).all()
    assert tq.device_status() == 0


@pytest.mark.parametrize("M,E", [(40, 16), (1200, 16), (300, 200)])
def test_experts_offsets_written_just_before(tq, M, E):
    """The kernel that writes the offsets, over other ones, and the product with nothing in
    between; every other time the offsets stay as they are."""
    import torch
    g = gen(M)
    N, K = 384, 512
    q, sx = tq.quant_act_f8(rows(g, M, K))
    Wq, sw = matrix(g, E, N, K)
    ws = tq.f8_workspace()
    ids = [torch.randint(0, E, (M, 1), generator=g, device="cuda", dtype=torch.int32) ** p % E for p in (1, 2, 3)]
    want = []
    for i in ids:
        off = tq.expert_sort(i, E)[0]
        torch.cuda.synchronize()
        want.append(tq.linear_f8_experts(q, sx, off, Wq, sw, ws, out="f32"))
    lists = tq.expert_sort(ids[0], E)
    got = []
    for i in range(24):
        off = tq.expert_sort(ids[i // 2 % 3], E, *lists)[0]
        got.append(tq.linear_f8_experts(q, sx, off, Wq, sw, ws, out="f32", Y=torch.empty(M, N, device="cuda")))
    for i, y in enumerate(got):
        assert torch.equal(y, want[i // 2 % 3])
    assert tq.device_status() == 0


@pytest.mark.parametrize("M", [3, 300])
@pytest.mark.parametrize("power", [-122, -136, -146])
def test_scales_whose_product_is_subnormal(tq, M, power):
    """sx * sw rounds to a multiple of 2^-149: off by 2^-150, on top of the usual bar, times
    a block's sum of magnitudes; Y itself is as coarse, and so is each block's addition."""
    import torch
    g = gen(-power)
    N, K = 140, 400
    q = torch.randint(0, 126, (M, K), generator=g, device="cuda", dtype=torch.uint8)
    w = torch.randint(0, 126, (N, K), generator=g, device="cuda", dtype=torch.uint8)
    sx = (1.0 + torch.rand(4, M, generator=g, device="cuda")) * 2.0 ** (power // 2)
    sw = (1.0 + torch.rand(2, 4, generator=g, device="cuda")) * 2.0 ** (power - power // 2)
    got = tq.linear_f8(q, sx, w, sw, tq.f8_workspace(), out="f32")
    want, S = ref.product(q, sx, w, sw)
    size = ref.decode(q) @ ref.decode(w).t()               # (no code is negative)
    bar = ref.product_bar(K, S, want, False) + 2.0 ** -150 * (size + 2 * 4 + 2)
    assert ((got.double() - want).abs() <= bar).all()
    assert tq.device_status() == 0


@pytest.mark.parametrize("M", [24, 700])
def test_product_in_a_graph_and_on_two_streams(tq, M):
    """A captured call replayed on new inputs, and two streams with a workspace each."""
    import torch
    g = gen(11)
    N, K = 896, 2048
    Wq, sw = matrix(g, N, K)
    x = [rows(g, M, K).contiguous() for _ in range(4)]
    ws = tq.f8_workspace()
    at = x[0].clone()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        q, sx = tq.quant_act_f8(at)
        tq.linear_f8(q, sx, Wq, sw, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tq.quant_act_f8(at, Xq=q, sx=sx)
        Y = tq.linear_f8(q, sx, Wq, sw, ws, out="f32")
    want = []
    for v in x:
        want.append(tq.linear_f8(*tq.quant_act_f8(v), Wq, sw, tq.f8_workspace(), out="f32"))
        at.copy_(v)
        graph.replay()
        assert torch.equal(Y, want[-1])
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for i in range(8):
        with torch.cuda.stream(streams[i % 2]):
            if i < 2:
                streams[i].ws = tq.f8_workspace()
            got.append(tq.linear_f8(*tq.quant_act_f8(x[i % 4]), Wq, sw, streams[i % 2].ws, out="f32"))
    torch.cuda.synchronize()
    for i, y in enumerate(got):
        assert torch.equal(y, want[i % 4])
    assert tq.device_status() == 0


@pytest.mark.parametrize("counts,N,K", [([16] * 64, 2048, 2048), ([33, 2, 40, 1] * 16, 2048, 1024),
                                        ([31, 33] * 4, 4096, 2048), ([300, 500, 7] * 8, 1024, 2048)])
def test_experts_many_tiles_again_and_again(tq, counts, N, K):
    """Several tiles a CTA, twenty times: the rounds of the stages and accumulators stay
    in step, and nothing depends on timing."""
    import torch
    g = gen(len(counts) + K)
    M = sum(counts)
    off = offsets_of(counts)
    q, sx = tq.quant_act_f8(rows(g, M, K))
    Wq, sw = matrix(g, len(counts), N, K)
    ws = tq.f8_workspace()
    first = tq.linear_f8_experts(q, sx, off, Wq, sw, ws, out="f32")
    a = 0
    for e, n in enumerate(counts):
        if e % 5 == 0:
            want, S = ref.product(q[a:a + n], sx[:, a:a + n], Wq[e], sw[e])
            check(first[a:a + n], want, S, K)
        a += n
    got = [tq.linear_f8_experts(q, sx, off, Wq, sw, ws, out="f32") for _ in range(20)]
    assert all(torch.equal(y, first) for y in got)
    assert tq.device_status() == 0
