"""Host refusals of the attention layer's entry points (no GPU): each names
its reason before any launch."""
import ctypes

import pytest

OK, NULL, SHAPE, BITS, MODE, OVERFLOW, ALIGN, WORKSPACE, CUDA, TIMEOUT, DEVICE, INDEX = range(12)
FAKE = 0x10000


@pytest.fixture(scope="module")
def L():
    import torch
    from dit_convrot_linear_gb300 import build, tq
    build.build()
    lib = tq.load()
    if torch.cuda.is_available():
        pytest.skip("refusal checks use fake device addresses: run them where no GPU is visible")
    return lib


def test_index_status_has_a_name():
    from dit_convrot_linear_gb300 import build, tq
    build.build()
    assert tq.load().tq_status_str(INDEX).decode().startswith("TQ_ERR_INDEX")
    assert tq.STATUS[INDEX] == "TQ_ERR_INDEX"


def norm(L, X=FAKE, M=4, K=896, ldx=896, R=FAKE, ldr=896, gamma=FAKE, eps=1e-6, H=FAKE, ldh=896, Y=FAKE, ldy=896,
         Xq=FAKE, sx=FAKE):
    return L.tq_rmsnorm_quant_act(X, M, K, ldx, R, ldr, gamma, eps, H, ldh, Y, ldy, Xq, sx, None)


def test_rmsnorm_refusals(L):
    assert norm(L) == DEVICE                                     # a valid call, and no GPU
    assert norm(L, R=None, H=None, Y=None) == DEVICE
    assert norm(L, Xq=None, sx=None) == DEVICE
    assert norm(L, M=0, X=None) == OK
    for kw, want in ((dict(X=None), NULL), (dict(gamma=None), NULL), (dict(Y=None, Xq=None, sx=None), NULL),
                     (dict(sx=None), NULL), (dict(Xq=None), NULL), (dict(M=-1), SHAPE), (dict(K=900), SHAPE),
                     (dict(K=16384 + 256, ldx=16640), SHAPE), (dict(ldx=888), SHAPE), (dict(ldr=888), SHAPE),
                     (dict(ldh=888), SHAPE), (dict(ldy=888), SHAPE), (dict(ldx=900), ALIGN), (dict(X=FAKE + 8), ALIGN),
                     (dict(R=FAKE + 2), ALIGN), (dict(H=FAKE + 2), ALIGN), (dict(Y=FAKE + 2), ALIGN),
                     (dict(gamma=FAKE + 4), ALIGN), (dict(Xq=FAKE + 4), ALIGN), (dict(sx=FAKE + 2), ALIGN),
                     (dict(eps=-1.0), MODE), (dict(eps=float("nan")), MODE), (dict(eps=float("inf")), MODE),
                     (dict(ldh=904), SHAPE),                     # H in X's place with another stride
                     (dict(M=1 << 60), OVERFLOW)):
        assert norm(L, **kw) == want, kw


def norm_tiled(L, M=4, K=896, at=FAKE, nbytes=1 << 30, sx=FAKE, **kw):
    d = dict(X=FAKE, ldx=896, R=None, ldr=0, gamma=FAKE, eps=1e-6, H=None, ldh=0)
    d.update(kw)
    return L.tq_rmsnorm_quant_act_tiled(d["X"], M, K, d["ldx"], d["R"], d["ldr"], d["gamma"], d["eps"], d["H"],
                                        d["ldh"], at, nbytes, sx, None)


def test_rmsnorm_tiled_refusals(L):
    assert norm_tiled(L) == DEVICE
    need = L.tq_act_tiled_bytes(4, 896)
    for kw, want in ((dict(at=None), NULL), (dict(sx=None), NULL), (dict(nbytes=need - 1), WORKSPACE),
                     (dict(at=FAKE + 128), ALIGN), (dict(gamma=None), NULL), (dict(eps=-1.0), MODE), (dict(K=31), SHAPE),
                     (dict(R=FAKE, ldr=8), SHAPE)):
        assert norm_tiled(L, **kw) == want, kw


def rope(L, X=FAKE, tokens=4, heads=2, dim=128, ldx=256, Y=FAKE * 2, ldy=256, spec=True, axis=None, **kw):
    from dit_convrot_linear_gb300 import tq
    d = dict(pos=FAKE, ldpos=4, inv_freq=FAKE, naxes=1, pairs=64, interleaved=0)
    d.update(kw)
    keep = None if axis is None else (ctypes.c_uint8 * len(axis))(*axis)
    s = tq.RopeSpecC(d["pos"], d["ldpos"], d["inv_freq"], None if keep is None else ctypes.addressof(keep), d["naxes"],
                     d["pairs"], d["interleaved"])
    return L.tq_rope(X, tokens, heads, dim, ldx, ctypes.addressof(s) if spec else None, Y, ldy, None)


def test_rope_refusals(L):
    assert rope(L) == DEVICE
    assert rope(L, Y=FAKE) == DEVICE                             # in place
    assert rope(L, axis=[0, 1] * 32, naxes=2) == DEVICE
    assert rope(L, tokens=0, X=None) == OK and rope(L, heads=0, X=None) == OK
    for kw, want in ((dict(spec=False), NULL), (dict(X=None), NULL), (dict(Y=None), NULL), (dict(pos=None), NULL),
                     (dict(inv_freq=None), NULL), (dict(tokens=-1), SHAPE), (dict(heads=-1), SHAPE), (dict(dim=0), SHAPE),
                     (dict(dim=12), SHAPE), (dict(dim=264, ldx=528, ldy=528), SHAPE), (dict(pairs=0), SHAPE),
                     (dict(pairs=65), SHAPE), (dict(naxes=0), SHAPE), (dict(naxes=5), SHAPE), (dict(interleaved=2), MODE),
                     (dict(ldx=248), SHAPE), (dict(ldy=248), SHAPE), (dict(ldx=260), ALIGN), (dict(X=FAKE + 8), ALIGN),
                     (dict(Y=FAKE + 8), ALIGN), (dict(Y=FAKE, ldy=264), SHAPE), (dict(ldpos=3), SHAPE),
                     (dict(pos=FAKE + 2), ALIGN), (dict(inv_freq=FAKE + 2), ALIGN),
                     (dict(axis=[0] * 63 + [1]), SHAPE), (dict(tokens=1 << 60, ldpos=1 << 60), OVERFLOW)):
        assert rope(L, **kw) == want, kw


def kv(**kw):
    from dit_convrot_linear_gb300 import tq
    d = dict(pool=FAKE, npages=10, page_size=16, heads=2, dim=128, table=FAKE, table_cols=4, ldt=4, kv_len=FAKE,
             q_start=FAKE, nseq=3, tokens=5)
    d.update(kw)
    return tq.KV4C(**d)


BAD_KV = [(dict(page_size=8), SHAPE), (dict(page_size=48), SHAPE), (dict(dim=96), SHAPE), (dict(heads=0), SHAPE),
          (dict(heads=1025), SHAPE), (dict(npages=-1), SHAPE), (dict(npages=1 << 31), SHAPE), (dict(nseq=-1), SHAPE),
          (dict(nseq=65537), SHAPE), (dict(tokens=-1), SHAPE), (dict(tokens=1 << 31), SHAPE), (dict(table_cols=-1), SHAPE),
          (dict(ldt=3), SHAPE), (dict(pool=None), NULL), (dict(table=None), NULL), (dict(kv_len=None), NULL),
          (dict(q_start=None), NULL), (dict(pool=FAKE + 8), ALIGN), (dict(table=FAKE + 2), ALIGN),
          (dict(kv_len=FAKE + 2), ALIGN), (dict(q_start=FAKE + 1), ALIGN), (dict(ldt=1 << 62), OVERFLOW)]


def test_kv4_page_bytes(L):
    assert L.tq_kv4_page_bytes(8, 128, 16) == 8 * (16 * 128 + 128)
    assert L.tq_kv4_page_bytes(1, 64, 128) == 8 * (16 * 64 + 128)
    assert L.tq_kv4_page_bytes(2, 256, 32) == 2 * 2 * (16 * 256 + 128)
    for bad in ((0, 128, 16), (2000, 128, 16), (1, 96, 16), (1, 128, 20), (-1, 128, 16)):
        assert L.tq_kv4_page_bytes(*bad) == 0
    assert L.tq_kv4_workspace_bytes() == 0                       # no GPU


def append(L, c=True, K=FAKE, ldk=256, V=FAKE, ldv=256, **kw):
    s = kv(**kw)
    return L.tq_kv4_append(ctypes.addressof(s) if c else None, K, ldk, V, ldv, None)


def read(L, c=True, K=FAKE, ldk=256, V=FAKE, ldv=256, **kw):
    s = kv(**kw)
    return L.tq_kv4_read(ctypes.addressof(s) if c else None, K, ldk, V, ldv, None)


@pytest.mark.parametrize("call", [append, read])
def test_append_and_read_refusals(L, call):
    assert call(L) == DEVICE
    assert call(L, tokens=0, K=None) == OK and call(L, nseq=0, pool=None) == OK
    assert call(L, c=False) == NULL
    for kw, want in BAD_KV + [(dict(ldk=248), SHAPE), (dict(ldv=248), SHAPE), (dict(ldk=260), ALIGN),
                              (dict(K=FAKE + 2), ALIGN), (dict(V=FAKE + 2), ALIGN), (dict(K=None, V=None), NULL)]:
        assert call(L, **kw) == want, kw
    assert append(L, K=None) == NULL and append(L, V=None) == NULL
    assert read(L, K=None) == DEVICE and read(L, V=None) == DEVICE


def attend(L, c=True, Q=FAKE, hq=8, ldq=1024, max_q=1, scale=0.1, causal=1, window=0, O=FAKE * 2, ldo=1024, lse=None,
           ws=FAKE, wb=1 << 40, **kw):
    s = kv(**kw)
    return L.tq_kv4_attention(ctypes.addressof(s) if c else None, Q, hq, ldq, max_q, scale, causal, window, O, ldo, lse,
                              ws, wb, None)


def test_attention_refusals(L):
    assert attend(L) == DEVICE and attend(L, O=FAKE, lse=FAKE) == DEVICE
    assert attend(L, tokens=0, Q=None) == OK
    assert attend(L, c=False) == NULL
    for kw, want in BAD_KV + [
            (dict(Q=None), NULL), (dict(O=None), NULL), (dict(hq=0), SHAPE), (dict(hq=1), SHAPE), (dict(hq=7), SHAPE),
            (dict(hq=130, ldq=130 * 128, ldo=130 * 128), SHAPE), (dict(ldq=1016), SHAPE), (dict(ldo=1016), SHAPE),
            (dict(ldq=1028), ALIGN), (dict(Q=FAKE + 8), ALIGN), (dict(O=FAKE + 8), ALIGN), (dict(O=FAKE, ldo=1032), SHAPE),
            (dict(max_q=0), SHAPE), (dict(window=-1), SHAPE), (dict(causal=2), MODE), (dict(scale=0.0), MODE),
            (dict(scale=-1.0), MODE), (dict(scale=float("nan")), MODE), (dict(scale=float("inf")), MODE),
            (dict(lse=FAKE + 2), ALIGN), (dict(ws=None), WORKSPACE), (dict(ws=FAKE + 128), ALIGN),
            (dict(tokens=1 << 30), OVERFLOW)]:
        assert attend(L, **kw) == want, kw


def test_binding_checks_tensors():
    """The binding refuses what the C ABI cannot see."""
    import torch
    from dit_convrot_linear_gb300 import build, tq
    build.build()
    with pytest.raises(ValueError):
        tq.KV4Cache(4, 16, 2, 96)
    x = torch.zeros(4, 896, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        tq.rmsnorm(x, torch.zeros(896))                          # not on the GPU
    with pytest.raises(ValueError):
        tq.RopeSpec(torch.zeros(4))
