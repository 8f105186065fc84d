"""The 4-bit cache and attention over it where a call can go wrong quietly:
scores with a large common part, padded page tables, bad pages among many
sequences, token scales far below their block's largest or not finite.
Against the 64-bit model on the GPU's own cache bytes."""
import numpy as np
import pytest

import kv4_ref as ref
from test_gpu_kv4 import INDEX, World, dev32, f64, rows

pytestmark = pytest.mark.gpu


def laid(tq, seqs, dim, codes_k, scales_k, codes_v, scales_v, heads=1, page=16):
    """A World whose sequences hold the given codes [heads, length, dim] and
    scales [heads, length] (one set for all)."""
    import torch
    w = World(tq, seqs, heads, dim, page, seed=1, fill=False, noise=False)
    pool = np.zeros((w.npages, heads, page // 16, ref.block_bytes(dim)), dtype=np.uint8)
    for b, (n, _) in enumerate(seqs):
        w._store(pool, b, codes_k[:, :n], scales_k[:, :n], 0)
        w._store(pool, b, codes_v[:, :n], scales_v[:, :n], 1)
    w.pool.copy_(torch.from_numpy(pool.reshape(-1)))
    return w


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("new,heads_q", [(1, 4), (5, 4), (20, 4), (50, 4), (300, 2)])
def test_scores_with_a_large_common_part(tq, dim, new, heads_q):
    """Scores of thousands that differ by a few: every key has 4 s in the one
    value that a constant query meets, s = 1, 1 + 2^-10 or 1 + 2^-9, all exact in
    fp16.  So a score's roundings are fp32's, below 2^-12 in the exponent (2^-24
    of 19000 and its factors), and those of a query's factor to fp16 are common to
    a row (2^-11 of the log sum).  Bars: weights and values rounded to fp16, a common factor of 2^-11 on
    differences of at most 32, 2^-6 a weight's for the others than the first;
    relative L2 2^-7 over the call, an element 2^-6 of its weighted values."""
    rng = np.random.default_rng(dim + new)
    n = 400
    ck = rng.integers(-7, 8, (1, n, dim))
    ck[..., 0] = 4
    sk = 1.0 + rng.integers(0, 3, (1, n)) / 1024.0
    cv, sv, _ = ref.quantise(rng.normal(size=(1, n, dim)), dim)
    w = laid(tq, [(n, new), (n - 130, new if new < 200 else 1)], dim, ck, sk, cv, sv)
    import torch
    size = np.array([45, -45, 94, -94, 188, -188, 400, -400]) * (1.0 if dim == 64 else 0.5)
    q = np.zeros((w.tokens, heads_q, dim))
    q += rng.choice(size, (w.tokens, heads_q))[..., None]
    Q = torch.from_numpy(q).cuda().bfloat16()
    O = torch.full_like(Q, float("nan"))
    lse = torch.empty(w.tokens, heads_q, device="cuda")
    tq.kv4_attention(w.batch, Q, 1.0, tq.kv4_workspace(), O=O, lse=lse)
    assert tq.device_status() == 0
    got, gl = f64(O), f64(lse)
    num = den = 0.0
    for b, (length, m) in enumerate(w.seqs):
        kc, vc, _, _ = w.cached(b)
        at = w.starts[b]
        qb = f64(Q[at:at + m])
        o, l, _, _ = ref.attend(qb, kc, vc, length, m, 1.0, True, 0)
        d = np.abs(got[at:at + m] - o)
        assert np.all(d <= 2.0 ** -8 * np.abs(o) + 2.0 ** -6 * np.abs(vc).sum(-1).max() / np.sqrt(dim))
        assert np.all(np.abs(gl[at:at + m] - l) <= 2.0 ** -10 * np.abs(l))
        num += float((d ** 2).sum())
        den += float((o ** 2).sum())
    assert num <= (2.0 ** -7) ** 2 * den, (num / den) ** 0.5


def test_page_table_with_wide_rows(tq):
    """A table that is part of a wider one gives the dense table's results; an
    expanded one is refused before anything runs."""
    import torch
    w = World(tq, [(100, 2), (33, 1), (70, 5)], 2, 64, 16, seed=60)
    Q = rows(w.tokens, 4, 64, 61, outliers=False)
    wide = torch.full((3, w.cols + 5), -1, dtype=torch.int32, device="cuda")
    wide[:, 2:2 + w.cols] = w.tab
    b = tq.KV4Batch(w.cache, wide[:, 2:2 + w.cols], w.lens, dev32(w.starts), w.tokens, 5)
    w.batch.max_q = 5
    assert torch.equal(tq.kv4_attention(b, Q, 0.1, tq.kv4_workspace()), tq.kv4_attention(w.batch, Q, 0.1, tq.kv4_workspace()))
    assert tq.device_status() == 0
    with pytest.raises(ValueError):
        tq.KV4Batch(w.cache, w.tab[:1].expand(3, w.cols), w.lens, dev32(w.starts), w.tokens, 5)


@pytest.mark.parametrize("bad", [7, 300, 511, 580])
def test_bad_page_among_many_sequences(tq, bad):
    """A page outside the pool is reported whichever of 600 sequences has it and
    whichever part of the GPU meets it, when written and when read."""
    w = World(tq, [(16, 2)] * 600, 8, 64, 16, seed=70, fill=False, noise=False)
    kv = rows(w.tokens, 16, 64, 71)
    tq.kv4_append(w.batch, kv[:, :8], kv[:, 8:])
    assert tq.device_status() == 0
    w.tab[bad, 0] = w.npages
    tq.kv4_append(w.batch, kv[:, :8], kv[:, 8:])
    assert tq.device_status() == INDEX and tq.device_status() == 0
    K, V = tq.kv4_read(w.batch)
    assert tq.device_status() == INDEX and tq.device_status() == 0
    gone = slice(2 * bad, 2 * bad + 2)
    assert not K[gone].any() and not V[gone].any() and int((K != 0).any(2).all(1).sum()) == w.tokens - 2


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("new,heads_q", [(6, 4), (80, 1), (150, 2)])
def test_scales_far_below_their_blocks_largest(tq, dim, new, heads_q):
    """Rows that see themselves alone, their scales 2^0 .. 2^-16 of their block's
    largest: the output is the value, the log sum the score.  Every rounding is
    within 2^-11 of what it rounds, however small that is beside its block: a
    key's scale, its product with the code and the query 3 x 2^-11 of the score, a
    value's two and the weight's 3 x 2^-11 and half a bf16 step (2^-8)."""
    import torch
    rng = np.random.default_rng(dim + new)
    n = new
    # one code a token and the query's rotated values all alike, so that a code's
    # error is the score's
    ck = np.broadcast_to(rng.integers(1, 8, (1, n, 1)) * rng.choice([-1, 1], (1, n, 1)), (1, n, dim)).copy()
    cv = rng.integers(-7, 8, (1, n, dim))
    sk, sv = (2.0 ** -rng.integers(0, 17, (1, n)) * rng.uniform(1, 2, (1, n)) for _ in range(2))
    sk[:, ::16], sv[:, ::16] = 1.0, 1.5
    sk, sv = sk.astype(np.float32).astype(np.float64), sv.astype(np.float32).astype(np.float64)
    w = laid(tq, [(n, new)], dim, ck, sk, cv, sv)
    q = np.zeros((w.tokens, heads_q, dim))
    q[..., 0] = 8.0
    Q = torch.from_numpy(q).cuda().bfloat16()
    O = torch.full_like(Q, float("nan"))
    lse = torch.empty(w.tokens, heads_q, device="cuda")
    tq.kv4_attention(w.batch, Q, 1.0, tq.kv4_workspace(), window=1, O=O, lse=lse)
    assert tq.device_status() == 0
    kc, vc, _, _ = w.cached(0)
    score = (kc[0] @ (f64(Q[0, 0]) @ ref.hadamard(dim)))[:, None]
    assert np.all(np.abs(f64(lse) - score) <= 3 * 2.0 ** -11 * np.abs(score) * 1.01 + 2.0 ** -20)
    want = (vc[0] @ ref.hadamard(dim))[:, None]
    bar = 2.0 ** -8 * np.abs(want) + 3 * 2.0 ** -11 * 1.01 * np.abs(vc[0]).sum(-1)[:, None, None] / np.sqrt(dim)
    assert np.all(np.abs(f64(O) - want) <= bar)
    # a call's rows as a whole: roundings of either sign, half of the worst at most
    num, den = ((f64(O) - want) ** 2).sum((1, 2)), (want ** 2).sum((1, 2)) * heads_q
    assert np.all(num <= (2.0 ** -8) ** 2 * den), np.sqrt(num / den).max()


def with_scale(w, b, pos, k, v):
    """The cache's bytes with other scales at a position of a sequence."""
    blocks = w.bytes().copy()
    at = 16 * w.dim + 4 * (pos % 16)
    blk = blocks[w.table[b, pos // w.page], :, pos % w.page // 16]
    for x, o in ((k, 0), (v, 64)):
        if x is not None:
            blk[:, at + o:at + o + 4] = np.array([x], np.float32).view(np.uint8)
    return blocks.reshape(-1)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new,heads_q", [(3, 2), (12, 2), (40, 4)])
@pytest.mark.parametrize("side", ["k", "v"])
@pytest.mark.parametrize("what", [float("nan"), float("inf")])
def test_a_scale_that_is_not_finite_where_some_rows_see_it(tq, dim, new, heads_q, side, what):
    """The rows that do not see such a token give the bits that they give where its
    scales are zero, though it lies in a tile that others of them see."""
    import torch
    n = 200
    w = World(tq, [(n, new), (50, new)], 1, dim, 16, seed=80)
    Q = rows(2 * new, heads_q, dim, 82, outliers=False)
    at = n - new // 2 - 1                                    # seen by the last new // 2 + 1 rows
    zero, odd = with_scale(w, 0, at, 0.0, 0.0), with_scale(w, 0, at, *((what, None) if side == "k" else (None, what)))
    outs = []
    for pool in (zero, odd):
        w.pool.copy_(torch.from_numpy(pool))
        lse = torch.zeros(2 * new, heads_q, device="cuda")
        outs.append((tq.kv4_attention(w.batch, Q, dim ** -0.5, tq.kv4_workspace(), lse=lse), lse))
    assert tq.device_status() == 0
    for a, b in zip(*outs):
        blind = torch.ones(2 * new, dtype=torch.bool, device="cuda")
        blind[new - new // 2 - 1:new] = False
        assert a.isfinite().all() and torch.equal(a[blind], b[blind])


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new,heads_q,n", [(3, 2, 200), (12, 2, 200), (40, 4, 200), (1, 4, 9000), (40, 4, 9000)])
@pytest.mark.parametrize("side", ["q", "k", "v"])
@pytest.mark.parametrize("what", [float("nan"), float("inf")])
def test_what_is_not_finite_shows_in_the_rows_that_see_it(tq, dim, new, heads_q, n, side, what):
    """NaN in the outputs and log sums of a query that is not finite, and of the
    rows that see a token whose key's scale is NaN or whose value's is not finite
    (whole row tiles and such as are cut into parts); every other row as it is without."""
    import torch
    w = World(tq, [(n, new), (50, new)], 1, dim, 64, seed=80)
    Q = rows(2 * new, heads_q, dim, 82, outliers=False)
    at = n - new // 2 - 1                                    # seen by the last new // 2 + 1 rows
    hit = torch.zeros(2 * new, heads_q, dtype=torch.bool, device="cuda")
    if side == "q":
        zero = odd = w.bytes().reshape(-1).copy()
        hit[0, 1] = True
    else:
        zero, odd = with_scale(w, 0, at, 0.0, 0.0), with_scale(w, 0, at, *((np.nan, None) if side == "k" else (None, what)))
        hit[new - new // 2 - 1:new] = True
    outs = []
    for pool, x in ((zero, 0.25), (odd, what)):
        w.pool.copy_(torch.from_numpy(pool))
        if side == "q":
            Q[0, 1, 7] = x
        lse = torch.zeros(2 * new, heads_q, device="cuda")
        outs.append((tq.kv4_attention(w.batch, Q, dim ** -0.5, tq.kv4_workspace(), lse=lse), lse))
    assert tq.device_status() == 0
    for a, b in zip(*outs):
        assert a.isfinite().all() and b[hit].isnan().all() and torch.equal(a[~hit], b[~hit])


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("count", [40, 5000])
def test_rows_that_are_not_finite_are_stored_as_such(tq, dim, count):
    """NaN or infinities in a head's row (written by rows and by blocks): its
    scale is NaN, it reads as NaN, every other row is as it is without."""
    w = World(tq, [(count, count), (33, 0)], 2, dim, 16, seed=83, fill=False, noise=False)
    kv = rows(w.tokens, 4, dim, 84)
    hit = {(3, 0): [np.nan], (20, 1): [np.inf], (21, 2): [-np.inf, np.inf], (count - 1, 3): [np.nan, np.inf]}
    for t, c in hit:
        kv[t, c] = 0
    tq.kv4_append(w.batch, kv[:, :2], kv[:, 2:])
    before = tq.kv4_read(w.batch)
    for (t, c), x in hit.items():
        for i, v in enumerate(x):
            kv[t, c, 7 + 20 * i] = v
    tq.kv4_append(w.batch, kv[:, :2], kv[:, 2:])
    after = tq.kv4_read(w.batch)
    assert tq.device_status() == 0
    for t, c in hit:
        assert after[c // 2][t, c % 2].isnan().all()
        after[c // 2][t, c % 2] = 0
        blk = w.bytes()[w.table[0, t // 16], c % 2, 0]
        assert np.isnan(blk[16 * dim:].copy().view(np.float32)[t % 16 + 16 * (c // 2)])
    assert all((a == b).all() for a, b in zip(after, before))
