"""The 4-bit cache on the GPU: appending and reading back, and attention over
it, against the 64-bit model of tests/kv4_ref.py on the GPU's own cache bytes.

Bars, set before the first run:
  - codes equal the 64-bit ones but where the rotated value over its scale lies
    within 2^-15 of a rounding boundary (|v / s| <= 7.5; the fp32 butterfly of
    at most 8 stages is within 2^-20 of the row's largest value, 7 times 2^-20
    in units of s, the scale itself within 2^-20 too), there by one; scales
    within 2^-20;
  - values read back: half a bf16 step (2^-8 of the value) plus 2^-18 of the
    row's largest rotated magnitude times sqrt(dim);
  - attention: kv4_ref.attend's bound plus half a bf16 step, element by
    element, and relative L2 at most 2^-8 over a call.
"""
import ctypes

import numpy as np
import pytest

import kv4_ref as ref
from helpers import to_np

pytestmark = pytest.mark.gpu

INDEX, TIMEOUT = 11, 9


def dev32(a):
    import torch
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


class World:
    """A cache with sequences of the given (length, new rows), its pages in a
    random order, filled with normal keys and values by the 64-bit model (or
    left as it is, noise in every byte, with fill=False)."""

    def __init__(self, tq, seqs, heads=2, dim=128, page=16, seed=0, fill=True, spare=2, noise=True, vspread=0.0,
                 order=None):
        import torch
        self.tq, self.seqs, self.heads, self.dim, self.page = tq, seqs, heads, dim, page
        rng = np.random.default_rng(seed)
        need = [-(-max(n, 0) // page) for n, _ in seqs]
        self.npages = sum(need) + spare
        self.cols = max(1, max(need))
        order = rng.permutation(self.npages) if order is None else order
        self.table = np.full((len(seqs), self.cols), 2 ** 30, dtype=np.int64)     # unused entries name no page
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        shape = (self.npages, heads, page // 16)
        blk = ref.block_bytes(dim)
        # unused places hold noise: any code, and scales that are NaN or infinite
        pool = rng.integers(0, 256, shape + (blk,), dtype=np.uint8)
        pool[..., 16 * dim:] = np.frombuffer(np.array([np.nan, np.inf] * 16, np.float32).tobytes(), np.uint8) \
            if noise else 0
        if fill:
            for b, (length, _) in enumerate(seqs):
                if length <= 0:
                    continue
                for v in (0, 1):
                    x = rng.normal(size=(heads, length, dim))
                    if v and vspread:
                        x *= 2.0 ** rng.uniform(-vspread, vspread, size=(heads, length, 1))
                    c, s, _ = ref.quantise(x, dim)
                    self._store(pool, b, c, s, v)
        self.pool = torch.from_numpy(pool.reshape(-1)).cuda()
        self.cache = tq.KV4Cache(self.npages, page, heads, dim, pool=self.pool)
        self.lens = dev32([n for n, _ in seqs])
        self.starts = np.concatenate([[0], np.cumsum([n for _, n in seqs])])
        self.tokens = int(self.starts[-1])
        self.tab = dev32(self.table)
        self.batch = tq.KV4Batch(self.cache, self.tab, self.lens, dev32(self.starts), self.tokens,
                                 max(1, max(n for _, n in seqs)))

    def _store(self, pool, b, codes, scales, v):
        dim = self.dim
        for t in range(codes.shape[1]):
            blk = pool[self.table[b, t // self.page], :, t % self.page // 16]
            r = t % 16
            u = (codes[:, t] + 8).astype(np.uint8)
            byte = u[:, 0::2] | (u[:, 1::2] << 4)
            if v:
                at = 8 * dim + (r // 2) * dim + (r % 2) * 2
                for k in range(dim // 4):
                    blk[:, at + 4 * k:at + 4 * k + 2] = byte[:, 2 * k:2 * k + 2]
            else:
                blk[:, r * dim // 2:(r + 1) * dim // 2] = byte
            at = 16 * dim + 64 * v + 4 * r
            blk[:, at:at + 4] = np.ascontiguousarray(scales[:, t].astype(np.float32)).view(np.uint8).reshape(-1, 4)

    def bytes(self):
        return ref.pool_blocks(to_np(self.pool), self.npages, self.heads, self.dim, self.page)

    def cached(self, b):
        return ref.sequence(self.bytes(), self.table[b], max(0, self.seqs[b][0]), self.page)


def rows(tokens, heads, dim, seed, outliers=True):
    import torch
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(tokens, heads, dim))
    if outliers:
        x[..., 3] *= 30.0
    return torch.from_numpy(x).cuda().bfloat16()


# ------------------------------------------------------------ append and read

@pytest.mark.parametrize("dim,page,heads", [(64, 16, 2), (128, 16, 8), (128, 64, 1), (256, 32, 3), (128, 128, 2)])
@pytest.mark.parametrize("many", [0, 1])
def test_append_and_read(tq, dim, page, heads, many):
    """Rows on their own, and by blocks (where they are many)."""
    seqs = [(1, 1), (37, 5), (16, 16), (129, 129), (200, 1), (0, 2), (33, 0)]
    if many:
        seqs += [(1500, 1400), (2001, 2001), (7, 9), (4000 // heads, 3990 // heads), (1000, 1000), (77, 60)]
    w = World(tq, seqs, heads, dim, page, seed=dim + page)
    kv = rows(w.tokens, 2 * heads, dim, 5)
    kv[3] = 0                                               # a row of zeros
    before = w.bytes().copy()
    tq.kv4_append(w.batch, kv[:, :heads], kv[:, heads:])    # strided: side by side in a token's row
    assert tq.device_status() == 0
    after = w.bytes()
    got_k, got_v = tq.kv4_read(w.batch)
    touched = np.zeros(before.shape, dtype=bool)
    for b, (length, new) in enumerate(seqs):
        for i in range(new):
            t, pos = w.starts[b] + i, length - new + i
            if pos < 0:
                assert not got_k[t].any() and not got_v[t].any()
                continue
            blk = (w.table[b, pos // page], slice(None), pos % page // 16)
            r = pos % 16
            k, v, sk, sv = ref.unpack(after[blk], dim)
            for x, c, s, out in ((kv[t, :heads], k[:, r], sk[:, r], got_k[t]), (kv[t, heads:], v[:, r], sv[:, r], got_v[t])):
                rc, rs, rt = ref.quantise(f64(x), dim)
                assert np.all(np.abs(s - rs) <= 2.0 ** -20 * rs)
                near = np.abs(np.abs(rt - np.floor(rt)) - 0.5) < 2.0 ** -15
                assert np.all((c == rc) | (near & (np.abs(c - rc) == 1)))
                want = (c * s[:, None]) @ ref.hadamard(dim)
                bar = 2.0 ** -8 * np.abs(want) + 2.0 ** -18 * 7 * s[:, None] * np.sqrt(dim)
                assert np.all(np.abs(f64(out) - want) <= bar)
            touched[blk + (slice(r * dim // 2, (r + 1) * dim // 2),)] = True
            at = 8 * dim + (r // 2) * dim + (r % 2) * 2
            for k4 in range(dim // 4):
                touched[blk + (slice(at + 4 * k4, at + 4 * k4 + 2),)] = True
            for s0 in (0, 64):
                touched[blk + (slice(16 * dim + s0 + 4 * r, 16 * dim + s0 + 4 * r + 4),)] = True
    assert np.array_equal(before[~touched], after[~touched])   # nothing beside the rows' own bytes
    assert tq.device_status() == 0


def test_read_whole_sequences_and_one_side(tq):
    import torch
    w = World(tq, [(70, 70), (5, 5)], heads=2, dim=128, page=32, seed=3)
    K = torch.full((75, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    V = torch.empty_like(K)
    tq.kv4_read(w.batch, K=K, V=V)
    for b, at in ((0, 0), (1, 70)):
        kc, vc, _, _ = w.cached(b)
        n = kc.shape[1]
        for out, c in ((K, kc), (V, vc)):
            want = np.moveaxis(c @ ref.hadamard(128), 0, 1)
            assert np.all(np.abs(f64(out[at:at + n]) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -15)
    K2 = torch.full_like(K, 7.0)
    L = tq.lib()
    assert L.tq_kv4_read(w.batch._p, K2.data_ptr(), 256, None, 0, torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(K2, K)


def test_append_bad_page_and_lengths_are_left_out(tq):
    """A page number outside the pool, a length above the table's and a row
    range outside the call: their rows are left out, the others written, and
    the status says so once."""
    import torch
    w = World(tq, [(20, 20), (20, 20), (4, 4)], heads=1, dim=128, page=16, seed=4)
    kv = rows(w.tokens, 2, 128, 6)
    before = w.bytes().copy()
    good = w.tab.clone()
    w.tab[0, 1] = w.npages                       # rows 16 .. 19 of sequence 0
    w.lens[2] = -5
    tq.kv4_append(w.batch, kv[:, :1], kv[:, 1:])
    assert tq.device_status() == INDEX and tq.device_status() == 0
    after = w.bytes()
    p0, p1 = w.table[0, 0], w.table[0, 1]
    assert not np.array_equal(before[p0], after[p0]) and np.array_equal(before[p1], after[p1])
    assert np.array_equal(before[w.table[2, 0]], after[w.table[2, 0]])
    K, V = tq.kv4_read(w.batch, K=torch.ones(w.tokens, 1, 128, dtype=torch.bfloat16, device="cuda"))
    assert tq.device_status() == INDEX
    assert not K[16:20].any() and K[:16].any(dim=2).all()
    w.tab.copy_(good)
    # a row range past the call's rows is taken as empty
    st = dev32([0, 20, 40, w.tokens + 1])
    w.lens[2] = 4
    b = tq.KV4Batch(w.cache, w.tab, w.lens, st, w.tokens, 20)
    tq.kv4_append(b, kv[:, :1], kv[:, 1:])
    assert tq.device_status() == INDEX and tq.device_status() == 0


def test_long_append_bad_page_and_more_rows_than_tokens(tq):
    """The same for calls of many rows: a page outside the pool, and a sequence
    with more rows than tokens (its first ones are before position 0)."""
    import torch
    w = World(tq, [(2500, 2500), (40, 700), (333, 333)], heads=4, dim=128, page=32, seed=40)
    kv = rows(w.tokens, 8, 128, 41)
    before = w.bytes().copy()
    w.tab[0, 7] = -3                             # rows 224 .. 255 of sequence 0
    tq.kv4_append(w.batch, kv[:, :4], kv[:, 4:])
    assert tq.device_status() == INDEX and tq.device_status() == 0
    after = w.bytes()
    lost = w.table[0, 7]
    assert np.array_equal(before[lost], after[lost])
    fill = torch.ones(w.tokens, 4, 128, dtype=torch.bfloat16, device="cuda")
    K, V = tq.kv4_read(w.batch, K=fill.clone(), V=fill.clone())
    assert tq.device_status() == INDEX
    for out, x in ((K, kv[:, :4]), (V, kv[:, 4:])):
        assert not out[224:256].any() and out[:224].any(dim=2).all() and out[256:2500].any(dim=2).all()
        assert not out[2500:3160].any() and out[3160:].any(dim=2).all()
        # 4-bit rounding leaves about 0.1 of a normal row
        keep = np.r_[0:224, 256:2500, 3160:w.tokens]
        d = f64(out)[keep] - f64(x)[keep]
        assert (d ** 2).sum() <= 0.2 ** 2 * (f64(x)[keep] ** 2).sum()


# ------------------------------------------------------------------ attention

def check(tq, w, heads_q, causal=True, window=0, seed=0, scale=None, Q=None, max_q=None, widened=False, l2=True):
    import torch
    dim = w.dim
    scale = dim ** -0.5 if scale is None else scale
    Q = rows(w.tokens, heads_q, dim, seed + 100, outliers=False) if Q is None else Q
    if max_q is not None:
        w.batch.max_q = max_q
    ws = tq.kv4_workspace()
    O = torch.full((w.tokens, heads_q, dim), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((w.tokens, heads_q), float("nan"), dtype=torch.float32, device="cuda")
    tq.kv4_attention(w.batch, Q, scale, ws, causal=causal, window=window, O=O, lse=lse)
    assert tq.device_status() == 0
    O2 = torch.empty_like(O)
    tq.kv4_attention(w.batch, Q, scale, ws, causal=causal, window=window, O=O2)   # the workspace is ready again
    assert torch.equal(O, O2)
    got, gl = f64(O), f64(lse)
    num = den = 0.0
    for b, (length, new) in enumerate(w.seqs):
        if new == 0:
            continue
        kc, vc, _, _ = w.cached(b) if length else (np.zeros((w.heads, 0, dim)),) * 2 + (None, None)
        at = w.starts[b]
        o, l, eo, el = ref.attend(f64(Q[at:at + new]), kc, vc, length, new, scale, causal, window, widened)
        d = np.abs(got[at:at + new] - o)
        assert np.all(d <= 2.0 ** -8 * np.abs(o) * (1 + 2.0 ** -8) + eo[..., None] * (1 + 2.0 ** -8)), \
            f"sequence {b}: {np.nanmax(d)}"
        gb = gl[at:at + new]
        assert np.array_equal(np.isneginf(gb), np.isneginf(l))
        fin = np.isfinite(l)
        assert np.all(np.abs(gb[fin] - l[fin]) <= el[fin])
        num += float((d ** 2).sum())
        den += float((o ** 2).sum())
    assert not l2 or num <= (2.0 ** -8) ** 2 * den or den == 0.0
    return O, lse


MIXED = [(1, 1), (31, 1), (32, 1), (33, 1), (0, 1), (500, 1), (1037, 1), (64, 0), (16, 1)]


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads,heads_q", [(2, 2), (2, 14), (1, 8), (2, 24), (1, 64)])
def test_decode_mixed_lengths(tq, dim, heads, heads_q):
    check(tq, World(tq, MIXED, heads, dim, 16, seed=dim + heads_q), heads_q)


@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_decode_page_sizes(tq, page):
    check(tq, World(tq, [(1, 1), (page, 1), (page + 1, 1), (3 * page - 1, 1), (777, 1)], 2, 128, page, seed=page), 8)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [0, 1, 40, 100000])
@pytest.mark.parametrize("dim,heads_q", [(128, 4), (64, 6), (256, 2)])
def test_several_rows_masks(tq, causal, window, dim, heads_q):
    seqs = [(5, 5), (90, 7), (300, 33), (0, 3), (64, 64), (2, 1)]
    check(tq, World(tq, seqs, 2, dim, 32, seed=window % 97 + dim), heads_q, causal, window)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads,heads_q,new", [(4, 16, 1), (4, 48, 1), (4, 16, 3), (3, 3, 1)])
def test_many_row_tiles(tq, dim, heads, heads_q, new):
    """Row tiles for every SM, a few much longer than the rest."""
    rng = np.random.default_rng(dim + heads_q)
    seqs = [(int(n), int(rng.integers(1, new + 1))) for n in rng.integers(0, 90, 24)]
    seqs[3], seqs[17] = (3000, new), (700, new)
    check(tq, World(tq, seqs, heads, dim, 32, seed=dim), heads_q)


@pytest.mark.parametrize("max_q", [1, 2, 8, 1000])
def test_max_q_is_a_hint(tq, max_q):
    """The same result, within the bars, whatever the hint says."""
    check(tq, World(tq, [(120, 9), (40, 2), (200, 1)], 2, 128, 16, seed=9), 6, max_q=max_q)


def test_rows_before_position_zero_see_nothing(tq):
    """More rows than tokens: the rows before position 0 give zeros and -inf."""
    w = World(tq, [(3, 9), (0, 4), (40, 40)], 1, 128, 16, seed=11)
    for causal in (True, False):
        O, lse = check(tq, w, 2, causal=causal)
        assert not O[:6].any() and bool((lse[:6] == -float("inf")).all())
        assert not O[9:13].any()


def test_one_long_sequence_and_many_sequences(tq):
    check(tq, World(tq, [(9000, 1)], 1, 128, 64, seed=12), 7)
    check(tq, World(tq, [(9001, 3), (5, 1)], 1, 64, 16, seed=13), 2)
    # more sequences than one scan step takes, some without rows or tokens
    rng = np.random.default_rng(1)
    seqs = [(int(n), int(n > 0 and m) or int(m > 1)) for n, m in zip(rng.integers(0, 70, 700), rng.integers(0, 3, 700))]
    check(tq, World(tq, seqs, 1, 64, 16, seed=14), 2)


@pytest.mark.parametrize("heads_q,new", [(8, 1), (16, 5)])
def test_sums_over_very_long_contexts(tq, heads_q, new):
    """Four sequences of 131072 tokens on the same pages, near-equal weights:
    outputs a hundredth of the values, of sums that must not carry the codes' bias
    of 8 along.  Relative L2 at most 0.0025: bf16's half step leaves 0.0017 at
    most (2^-9 / sqrt(3) of a value just above a power of two), weights rounded
    to fp16 2^-11 / sqrt(3)."""
    import torch
    heads, dim, page, n = 8, 128, 128, 131072
    rng = np.random.default_rng(50)
    np_ = n // page
    kc, vc = (np.clip(np.rint(rng.normal(size=(np_, heads, page // 16, 16, dim)) * 2.6), -7, 7).astype(np.int64)
              for _ in range(2))
    sk, sv = (rng.uniform(a, 2 * a, (np_, heads, page // 16, 16)).astype(np.float32) for a in (0.05, 0.25))
    pool = torch.from_numpy(ref.pack(kc, vc, sk, sv).reshape(-1)).cuda()
    cache = tq.KV4Cache(np_, page, heads, dim, pool=pool)
    tab = torch.arange(np_, dtype=torch.int32, device="cuda").expand(4, np_).contiguous()
    batch = tq.KV4Batch(cache, tab, dev32([n] * 4), dev32(np.arange(5) * new), 4 * new, new)
    Q = rows(4 * new, heads_q, dim, 51, outliers=False)
    O = f64(tq.kv4_attention(batch, Q, dim ** -0.5, tq.kv4_workspace()))
    assert tq.device_status() == 0
    H, q = ref.hadamard(dim), f64(Q)
    num = den = 0.0
    for h in range(heads):
        k = (kc[:, h] * sk[:, h, ..., None].astype(np.float64)).reshape(n, dim)
        v = (vc[:, h] * sv[:, h, ..., None].astype(np.float64)).reshape(n, dim)
        g = heads_q // heads
        for b in (0, 3):
            for i in range(new):
                x = (q[b * new + i, h * g:(h + 1) * g] @ H) @ k.T * dim ** -0.5
                x[:, n - new + i + 1:] = -np.inf
                w = np.exp(x - x.max(1, keepdims=True))
                o = (w / w.sum(1, keepdims=True)) @ v @ H
                num += ((O[b * new + i, h * g:(h + 1) * g] - o) ** 2).sum()
                den += (o ** 2).sum()
    assert num <= 0.0025 ** 2 * den, (num / den) ** 0.5


def test_value_scales_of_all_sizes(tq):
    """Values whose scales span 2^-20 .. 2^20 within a sequence, and all tiny."""
    check(tq, World(tq, [(300, 1), (90, 2)], 1, 128, 16, seed=15, vspread=20.0), 4)
    w = World(tq, [(100, 1)], 1, 128, 16, seed=16)
    blocks = w.bytes().copy()
    s = blocks[..., 16 * 128 + 64:].copy().view(np.float32)
    blocks[..., 16 * 128 + 64:] = (np.nan_to_num(s, posinf=0.0) * np.float32(2.0 ** -100)).view(np.uint8)
    import torch
    w.pool.copy_(torch.from_numpy(blocks.reshape(-1)))
    check(tq, w, 4)


def test_large_scores(tq):
    """Scores of hundreds (one position takes all the weight) and a late
    position above every earlier one (the running maximum rises to the end)."""
    import torch
    w = World(tq, [(600, 1), (600, 2)], 1, 128, 16, seed=17)
    Q = rows(w.tokens, 4, 128, 3, outliers=False) * 16
    O, _ = check(tq, w, 4, Q=Q, scale=1.0)
    assert torch.isfinite(O.float()).all()


def test_queries_of_extreme_size_and_zero(tq):
    w = World(tq, [(90, 1)] * 4, 1, 128, 16, seed=18)
    Q = rows(w.tokens, 2, 128, 4, outliers=False)
    Q[0] = 0
    Q[1] *= 1e-20
    Q[2] *= 1e-38
    check(tq, w, 2, Q=Q)


def test_zero_keys_and_values(tq):
    w = World(tq, [(90, 1)], 1, 128, 16, seed=19)
    import torch
    w.pool.copy_(torch.from_numpy(np.zeros(w.pool.numel(), dtype=np.uint8)))   # every code -8, every scale 0
    O, lse = check(tq, w, 2)
    assert not O.any()
    assert torch.allclose(lse, torch.full_like(lse, float(np.log(90))))


def test_strided_rows_in_place_and_another_stream(tq):
    """Queries as a slice of a fused projection's row, the output in their
    place, on a stream that is not the current one."""
    import torch
    w = World(tq, [(200, 2), (77, 3)], 2, 128, 16, seed=20)
    base = rows(w.tokens, 8 + 4, 128, 7, outliers=False)
    keep = base.clone()
    ws = tq.kv4_workspace()
    want = tq.kv4_attention(w.batch, keep[:, :8].contiguous(), 128 ** -0.5, ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    q = base[:, :8]
    tq.kv4_attention(w.batch, q, 128 ** -0.5, ws, O=q, stream=s)
    s.synchronize()
    assert torch.equal(base[:, :8], want) and torch.equal(base[:, 8:], keep[:, 8:])
    assert tq.device_status() == 0


def test_pool_past_32_bits(tq):
    """Pages beyond 4 GiB of the pool."""
    import torch
    heads, dim, page = 8, 128, 128
    pb = tq.kv4_page_bytes(heads, dim, page)
    npages = (5 << 30) // pb
    pool = torch.empty(npages * pb, dtype=torch.uint8, device="cuda")
    cache = tq.KV4Cache(npages, page, heads, dim, pool=pool)
    n = 300
    table = dev32([[npages - 1, npages - 5, npages // 2]])
    batch = tq.KV4Batch(cache, table, dev32([n]), dev32([0, n]), n, n)
    kv = rows(n, 2 * heads, dim, 8)
    tq.kv4_append(batch, kv[:, :heads], kv[:, heads:])
    K, V = tq.kv4_read(batch)
    Q = rows(n, heads, dim, 9, outliers=False)
    O = tq.kv4_attention(batch, Q, dim ** -0.5, tq.kv4_workspace())
    assert tq.device_status() == 0
    small = tq.KV4Cache(3, page, heads, dim)
    b2 = tq.KV4Batch(small, dev32([[2, 0, 1]]), dev32([n]), dev32([0, n]), n, n)
    tq.kv4_append(b2, kv[:, :heads], kv[:, heads:])
    K2, V2 = tq.kv4_read(b2)
    assert torch.equal(K, K2) and torch.equal(V, V2)
    assert torch.equal(O, tq.kv4_attention(b2, Q, dim ** -0.5, tq.kv4_workspace()))


def test_attention_bad_indices_are_left_out(tq):
    """A page outside the pool: its tokens are masked, the rest attended, and
    the status says so; a bad length or row range likewise."""
    import torch
    w = World(tq, [(100, 1), (40, 1)], 1, 128, 16, seed=21)
    Q = rows(w.tokens, 2, 128, 10, outliers=False)
    ws = tq.kv4_workspace()
    w.tab[0, 2] = -1                                 # positions 32 .. 47
    O = tq.kv4_attention(w.batch, Q, 128 ** -0.5, ws)
    assert tq.device_status() == INDEX and tq.device_status() == 0
    w.table[0, 2] = w.table[0, 1]
    kc, vc, _, _ = w.cached(0)
    keep = np.r_[0:32, 48:100]
    o, _, eo, _ = ref.attend(f64(Q[:1]), kc[:, keep], vc[:, keep], 84, 1, 128 ** -0.5, True, 0)
    assert np.all(np.abs(f64(O[:1]) - o) <= 2.0 ** -8 * np.abs(o) * 1.01 + eo[..., None] * 1.01)
    w.tab[0, 2] = int(w.table[0, 1])
    w.lens[0] = w.cols * 16 + 1                      # taken as the table's capacity
    tq.kv4_attention(w.batch, Q, 128 ** -0.5, ws)
    assert tq.device_status() == INDEX
    w.lens[0] = 100
    b = tq.KV4Batch(w.cache, w.tab, w.lens, dev32([1, 0, 2]), 2, 1)
    O = torch.full((2, 2, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    tq.kv4_attention(b, Q, 128 ** -0.5, ws, O=O)
    assert tq.device_status() == INDEX and tq.device_status() == 0


def test_append_then_attend_follows_the_unquantised_attention(tq):
    """The whole path on outlier channels: attention over the cache against
    attention over the unquantised keys and values.  4-bit rounding of a normal
    row leaves about 0.1 of it (a step of amax / 7, amax about 2.7 sigma at 128
    values, over sqrt(12)); over 400 positions a third of that: 0.2 is beyond
    it and far below what a misplaced token or axis leaves (about 1)."""
    import torch
    n, heads, hq, dim = 400, 2, 8, 128
    w = World(tq, [(n, n)], heads, dim, 16, seed=22, fill=False)
    kv = rows(n, 2 * heads, dim, 11)
    tq.kv4_append(w.batch, kv[:, :heads], kv[:, heads:])
    Q = rows(n, hq, dim, 12, outliers=False)
    O = f64(tq.kv4_attention(w.batch, Q, 0.02, tq.kv4_workspace()))
    k, v, q = f64(kv[:, :heads]), f64(kv[:, heads:]), f64(Q)
    num = den = 0.0
    for h in range(hq):
        x = 0.02 * q[:, h] @ k[:, h // 4].T
        x[np.triu_indices(n, 1)] = -np.inf
        p = np.exp(x - x.max(1, keepdims=True))
        o = (p / p.sum(1, keepdims=True)) @ v[:, h // 4]
        num += ((O[:, h] - o) ** 2).sum()
        den += (o ** 2).sum()
    assert num <= 0.2 ** 2 * den
    assert tq.device_status() == 0


def test_expired_wait_is_reported(tq):
    """A copy of the library whose attention stages expect 16 bytes that no
    copy brings, its waits limited to 2e6 cycles: the call ends, the status
    names the expiry once, nothing is written, and the product library's next
    call on the same context and workspace is right."""
    import torch
    from dit_convrot_linear_gb300 import build
    path = build.build_variant("kv4_expiry", ["TQ_TEST_UNSET_BYTES=16", "TQ_TEST_WAIT_CYCLES=2000000"],
                               ["k_kv4_attn.cu"])
    L = ctypes.CDLL(path)
    for name in ("tq_kv4_attention", "tq_device_status"):
        fn = getattr(L, name)
        fn.restype, fn.argtypes = tq.SIGNATURES[name]
    w = World(tq, [(700, 1), (20, 1)], 1, 128, 16, seed=23)
    Q = rows(w.tokens, 2, 128, 13, outliers=False)
    O = torch.zeros((w.tokens, 2, 128), dtype=torch.bfloat16, device="cuda")
    ws = tq.kv4_workspace()
    s = torch.cuda.current_stream().cuda_stream
    assert L.tq_kv4_attention(w.batch._p, Q.data_ptr(), 2, 256, 1, 0.1, 1, 0, O.data_ptr(), 256, None, ws.data_ptr(),
                              ws.numel(), s) == 0
    assert L.tq_device_status(s) == TIMEOUT and L.tq_device_status(s) == 0
    assert not O.any()
    got = tq.kv4_attention(w.batch, Q, 0.1, ws)
    assert torch.equal(got, tq.kv4_attention(w.batch, Q, 0.1, tq.kv4_workspace()))
    check(tq, w, 2)
