"""Attention over the 4-bit cache for tens of query rows a key/value head
(prompts, chunks of them, drafted tokens), against the 64-bit model on the GPU's
own cache bytes.  Bars, set before the first run: kv4_ref.attend's bound for
widened keys and values plus half a bf16 step, element by element, and relative
L2 at most 2^-8 over a call (the half step leaves 2^-9 / sqrt(3) / (1 - 2^-9)
of it, the roundings to fp16 about 2^-11 each, averaged over positions)."""
import ctypes

import numpy as np
import pytest

import kv4_ref as ref
from test_gpu_kv4 import INDEX, TIMEOUT, World, check, dev32, f64, rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page", [16, 64, 128])
@pytest.mark.parametrize("heads,heads_q,new", [(2, 8, 5), (1, 1, 128), (1, 1, 129), (2, 10, 7), (1, 8, 33), (1, 32, 9)])
def test_lengths_around_tiles(tq, dim, page, heads, heads_q, new):
    """One to several row tiles of 128 or 256 rows; contexts that end before, at
    and after a block, a half and a tile."""
    seqs = [(new, new), (127, new), (128, new), (129, 2), (145, new), (500, new), (0, 3), (64, 0), (250, 1)]
    check(tq, World(tq, seqs, heads, dim, page, seed=dim + page + new), heads_q, widened=True)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [0, 1, 40, 200, 100000])
@pytest.mark.parametrize("dim,heads_q", [(128, 4), (64, 12)])
def test_masks(tq, causal, window, dim, heads_q):
    """Rows without a position (before 0), windows within a block and over
    several tiles, rows that see the tokens after them."""
    seqs = [(50, 90), (700, 70), (300, 33), (0, 40), (64, 64), (2, 1)]
    O, lse = check(tq, World(tq, seqs, 2, dim, 32, seed=window % 97 + dim), heads_q, causal, window, widened=True)
    assert not O[:40].any() and bool((lse[:40] == -float("inf")).all())


@pytest.mark.parametrize("length,new,heads,heads_q", [(9001, 5, 1, 4), (5000, 40, 1, 8), (16, 17, 1, 1), (2500, 600, 2, 2)])
def test_row_tiles_in_parts(tq, length, new, heads, heads_q):
    """Few row tiles, cut along the positions and joined."""
    check(tq, World(tq, [(length, new)], heads, 128, 64, seed=length), heads_q, widened=True)


def test_many_sequences(tq):
    """Row tiles enough that a piece holds several, short and long, some empty;
    and more sequences than the many-row form takes."""
    rng = np.random.default_rng(2)
    for count, heads in ((192, 2), (256, 3), (257, 1)):
        seqs = [(int(n), int(m)) for n, m in zip(rng.integers(0, 300, count), rng.integers(0, 7, count))]
        seqs[5] = (2000, 20)
        check(tq, World(tq, seqs, heads, 64, 16, seed=count), 4 * heads, widened=True)


@pytest.mark.parametrize("max_q", [1, 3, 1000])
def test_max_q_is_a_hint(tq, max_q):
    check(tq, World(tq, [(320, 90), (40, 2), (200, 1)], 2, 128, 16, seed=9), 6, max_q=max_q, widened=True)


@pytest.mark.parametrize("new", [6, 50])
def test_value_scales_of_all_sizes(tq, new):
    """Values whose scales span 2^-20 .. 2^20 within a sequence, and all tiny."""
    import torch
    w = World(tq, [(300, new), (90, 2)], 1, 128, 16, seed=15, vspread=20.0)
    check(tq, w, 4, widened=True)
    for factor in (2.0 ** -100, 2.0 ** 100):
        w = World(tq, [(200, new)], 1, 128, 16, seed=16)
        blocks = w.bytes().copy()
        s = blocks[..., 16 * 128 + 64:].copy().view(np.float32)
        blocks[..., 16 * 128 + 64:] = (np.nan_to_num(s, posinf=0.0) * np.float32(factor)).view(np.uint8)
        w.pool.copy_(torch.from_numpy(blocks.reshape(-1)))
        check(tq, w, 4, widened=True)


@pytest.mark.parametrize("new", [6, 50])
def test_large_scores(tq, new):
    """Scores of hundreds: one position takes the weight, and the running maximum
    rises late.  No relative L2 here: keys rounded to fp16, all else exact, move a
    score of 500 by 2^-12 of it and leave 0.0052 of these outputs (new = 50),
    which the bound by element allows for."""
    import torch
    w = World(tq, [(600, new), (600, 2)], 1, 128, 16, seed=17)
    O, _ = check(tq, w, 4, Q=rows(w.tokens, 4, 128, 3, outliers=False) * 16, scale=1.0, widened=True, l2=False)
    assert torch.isfinite(O.float()).all()


def test_queries_of_extreme_size_and_zero(tq):
    w = World(tq, [(90, 10)] * 4, 1, 128, 16, seed=18)
    Q = rows(w.tokens, 2, 128, 4, outliers=False)
    Q[0] = 0
    Q[1] *= 1e-20
    Q[2] *= 1e-38
    check(tq, w, 2, Q=Q, widened=True)


@pytest.mark.parametrize("heads_q", [2, 16])
def test_zero_keys_and_values(tq, heads_q):
    import torch
    w = World(tq, [(290, 20)], 1, 128, 16, seed=19)
    w.pool.copy_(torch.from_numpy(np.zeros(w.pool.numel(), dtype=np.uint8)))   # every code -8, every scale 0
    O, lse = check(tq, w, heads_q, widened=True)
    assert not O.any()
    want = torch.log(torch.arange(271, 291, device="cuda", dtype=torch.float32))
    assert torch.allclose(lse, want[:, None].expand_as(lse))


def test_strided_rows_in_place_and_another_stream(tq):
    import torch
    w = World(tq, [(400, 30), (77, 12)], 2, 128, 16, seed=20)
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


def test_few_and_many_rows_share_a_workspace(tq):
    """One workspace for calls of both forms, in turn."""
    import torch
    a = World(tq, [(900, 1), (50, 1)], 2, 128, 16, seed=30)
    b = World(tq, [(900, 40), (50, 5)], 2, 128, 16, seed=31)
    ws = tq.kv4_workspace()
    qa, qb = rows(a.tokens, 8, 128, 1, outliers=False), rows(b.tokens, 8, 128, 2, outliers=False)
    oa, ob = (tq.kv4_attention(w.batch, q, 0.09, tq.kv4_workspace()) for w, q in ((a, qa), (b, qb)))
    for _ in range(3):
        assert torch.equal(tq.kv4_attention(a.batch, qa, 0.09, ws), oa)
        assert torch.equal(tq.kv4_attention(b.batch, qb, 0.09, ws), ob)
    assert tq.device_status() == 0


@pytest.mark.parametrize("seqs,heads,heads_q,dim", [
    ([(300, 300)], 8, 8, 128), ([(4096, 1024)], 4, 16, 128), ([(900, 33), (2000, 70), (64, 40)], 2, 4, 64),
    ([(3000, 5), (70, 3), (1500, 1)] * 6, 2, 8, 128), ([(2000, 1), (90, 1)] * 16, 4, 16, 256)])
def test_results_do_not_depend_on_timing(tq, seqs, heads, heads_q, dim):
    """The same call from cold caches, from an idle device and back to back, its
    results the same bits: no warp reads what another has yet to write."""
    import torch
    w = World(tq, seqs, heads, dim, 16, seed=60, fill=False, noise=False)
    full = np.array([n for n, _ in seqs])
    kv = rows(int(full.sum()), 2 * heads, dim, 61)
    tq.kv4_append(tq.KV4Batch(w.cache, w.tab, w.lens, dev32(np.concatenate([[0], full.cumsum()])), int(full.sum()),
                              int(full.max())), kv[:, :heads], kv[:, heads:])
    Q = rows(w.tokens, heads_q, dim, 62, outliers=False)
    ws, flush = tq.kv4_workspace(), torch.empty(400 << 20, dtype=torch.uint8, device="cuda")
    outs = []
    for i in range(18):
        if i % 3 == 0:
            flush.fill_(i)
        if i % 3 == 1:
            torch.cuda.synchronize()
        lse = torch.empty(w.tokens, heads_q, device="cuda")
        outs.append((tq.kv4_attention(w.batch, Q, dim ** -0.5, ws, lse=lse), lse))
    assert tq.device_status() == 0
    assert all(torch.equal(o, outs[0][0]) and torch.equal(x, outs[0][1]) for o, x in outs)


def test_bad_page_is_left_out(tq):
    """A page outside the pool: its tokens are masked for every row, the rest
    attended, and the status says so."""
    w = World(tq, [(300, 9), (40, 9)], 1, 128, 16, seed=21)
    Q = rows(w.tokens, 4, 128, 10, outliers=False)
    w.tab[0, 2] = -1                                 # positions 32 .. 47
    w.tab[0, 9] = w.npages                           # positions 144 .. 159
    O = tq.kv4_attention(w.batch, Q, 128 ** -0.5, tq.kv4_workspace())
    assert tq.device_status() == INDEX and tq.device_status() == 0
    kc, vc, _, _ = w.cached(0)
    keep = np.r_[0:32, 48:144, 160:300]
    o, _, eo, _ = ref.attend(f64(Q[:9]), kc[:, keep], vc[:, keep], len(keep), 9, 128 ** -0.5, True, 0, True)
    assert np.all(np.abs(f64(O[:9]) - o) <= 2.0 ** -8 * np.abs(o) * 1.01 + eo[..., None] * 1.01)


def test_expired_wait_is_reported(tq):
    """A copy of the library whose ring expects 16 bytes that no copy brings, its
    waits limited to 2e6 cycles: the call ends, the status names the expiry once,
    and the product library's next call on the same workspace is right."""
    import torch
    from dit_convrot_linear_gb300 import build
    path = build.build_variant("kv4_rows_expiry", ["TQ_TEST_UNSET_BYTES=16", "TQ_TEST_WAIT_CYCLES=2000000"],
                               ["k_kv4_attn_tc.cu"])
    L = ctypes.CDLL(path)
    for name in ("tq_kv4_attention", "tq_device_status"):
        fn = getattr(L, name)
        fn.restype, fn.argtypes = tq.SIGNATURES[name]
    w = World(tq, [(700, 9), (20, 9)], 1, 128, 16, seed=23)
    Q = rows(w.tokens, 4, 128, 13, outliers=False)
    O = torch.zeros((w.tokens, 4, 128), dtype=torch.bfloat16, device="cuda")
    ws = tq.kv4_workspace()
    s = torch.cuda.current_stream().cuda_stream
    assert L.tq_kv4_attention(w.batch._p, Q.data_ptr(), 4, 512, 9, 0.1, 1, 0, O.data_ptr(), 512, None, ws.data_ptr(),
                              ws.numel(), s) == 0
    assert L.tq_device_status(s) == TIMEOUT and L.tq_device_status(s) == 0
    got = tq.kv4_attention(w.batch, Q, 0.1, ws)
    assert torch.equal(got, tq.kv4_attention(w.batch, Q, 0.1, tq.kv4_workspace()))
    check(tq, w, 4, widened=True)
