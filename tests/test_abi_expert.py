"""Host refusals of the 8-bit floating-point products and of the experts' entry
points (no GPU): each names its reason before any launch."""
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


def refuses(call, cases):
    for kw, want in cases:
        assert call(**kw) == want, kw


def test_weights(L):
    def call(W=FAKE, N=4, K=896, ldw=896, codes=FAKE, scales=FAKE):
        return L.tq_quantize_weights_f8(W, N, K, ldw, codes, scales, None)
    assert call() == DEVICE and call(N=0, W=None) == OK and call(K=16, ldw=16) == DEVICE
    refuses(call, [(dict(W=None), NULL), (dict(codes=None), NULL), (dict(scales=None), NULL), (dict(N=-1), SHAPE),
                   (dict(K=0), SHAPE), (dict(K=24), SHAPE), (dict(K=65552, ldw=65552), SHAPE), (dict(ldw=888), SHAPE),
                   (dict(ldw=900), ALIGN), (dict(W=FAKE + 8), ALIGN), (dict(codes=FAKE + 8), ALIGN),
                   (dict(scales=FAKE + 2), ALIGN), (dict(N=1 << 60), OVERFLOW)])


def test_rows(L):
    def call(X=FAKE, R=4, K=896, ldx=896, rows=None, M=4, Xq=FAKE, sx=FAKE):
        return L.tq_quant_act_f8(X, R, K, ldx, rows, M, Xq, sx, None)
    assert call() == DEVICE and call(M=0, R=0) == OK and call(rows=FAKE, M=9) == DEVICE
    assert call(rows=FAKE, X=None, R=0) == DEVICE            # no row can be named but -1
    refuses(call, [(dict(X=None), NULL), (dict(Xq=None), NULL), (dict(sx=None), NULL), (dict(M=5), SHAPE),
                   (dict(M=-1, R=-1), SHAPE), (dict(R=-1, rows=FAKE), SHAPE), (dict(K=20), SHAPE), (dict(ldx=880), SHAPE),
                   (dict(ldx=900), ALIGN), (dict(X=FAKE + 2), ALIGN), (dict(Xq=FAKE + 8), ALIGN),
                   (dict(sx=FAKE + 1), ALIGN), (dict(rows=FAKE + 2), ALIGN),
                   (dict(rows=FAKE, M=1 << 31), OVERFLOW), (dict(rows=FAKE, R=1 << 60), OVERFLOW)])


def test_swiglu(L):
    def call(G=FAKE, ldg=512, U=FAKE, ldu=512, M=4, K=256, Xq=FAKE, sx=FAKE):
        return L.tq_swiglu_quant_act_f8(G, ldg, U, ldu, M, K, Xq, sx, None)
    assert call() == DEVICE and call(M=0, G=None) == OK
    refuses(call, [(dict(G=None), NULL), (dict(U=None), NULL), (dict(Xq=None), NULL), (dict(sx=None), NULL),
                   (dict(M=-1), SHAPE), (dict(K=8), SHAPE), (dict(ldg=255), SHAPE), (dict(ldu=248), SHAPE),
                   (dict(ldg=260), ALIGN), (dict(U=FAKE + 2), ALIGN), (dict(M=1 << 40), OVERFLOW)])


def product(L, experts=None, **kw):
    d = dict(Xq=FAKE, sx=FAKE, M=4, K=896, off=FAKE, Wq=FAKE, sw=FAKE, N=300, Y=FAKE, ytype=1, ldy=300, ws=FAKE,
             nbytes=1 << 40)
    d.update(kw)
    tail = (d["Wq"], d["sw"], d["N"], d["Y"], d["ytype"], d["ldy"], d["ws"], d["nbytes"], None)
    if experts is None:
        return L.tq_linear_f8(d["Xq"], d["sx"], d["M"], d["K"], *tail)
    return L.tq_linear_f8_experts(d["Xq"], d["sx"], d["M"], d["K"], d["off"], experts, *tail)


@pytest.mark.parametrize("experts", [None, 3])
def test_products(L, experts):
    def call(**kw):
        return product(L, **{"experts": experts, **kw})
    assert call() == DEVICE and call(M=0, Xq=None) == OK and call(N=0, Wq=None) == OK
    refuses(call, [(dict(Xq=None), NULL), (dict(sx=None), NULL), (dict(Wq=None), NULL), (dict(sw=None), NULL),
                   (dict(Y=None), NULL), (dict(M=-1), SHAPE), (dict(N=-1), SHAPE), (dict(K=900), SHAPE),
                   (dict(K=65536 + 16), SHAPE), (dict(ldy=299), SHAPE), (dict(ytype=2), MODE), (dict(ytype=-1), MODE),
                   (dict(Xq=FAKE + 8), ALIGN), (dict(Wq=FAKE + 8), ALIGN), (dict(sx=FAKE + 2), ALIGN),
                   (dict(sw=FAKE + 2), ALIGN), (dict(Y=FAKE + 1), ALIGN), (dict(ytype=0, Y=FAKE + 2), ALIGN),
                   (dict(ws=None), WORKSPACE), (dict(ws=FAKE + 128), ALIGN), (dict(M=1 << 31), OVERFLOW),
                   (dict(N=1 << 31, ldy=1 << 31), OVERFLOW)])
    if experts is not None:
        refuses(call, [(dict(off=None), NULL), (dict(off=FAKE + 2), ALIGN), (dict(experts=0), SHAPE),
                       (dict(experts=1025), SHAPE), (dict(experts=1024, N=1 << 22, ldy=1 << 22), OVERFLOW)])


def test_workspace_needs_a_device(L):
    assert L.tq_f8_workspace_bytes() == 0


def test_topk(L):
    def call(x=FAKE, t=1, T=4, E=64, ld=64, top=8, renorm=1, ids=FAKE, w=FAKE):
        return L.tq_expert_topk(x, t, T, E, ld, top, renorm, ids, w, None)
    assert call() == DEVICE and call(T=0, x=None) == OK and call(E=1024, ld=1024, top=32) == DEVICE
    refuses(call, [(dict(x=None), NULL), (dict(ids=None), NULL), (dict(w=None), NULL), (dict(t=2), MODE),
                   (dict(renorm=2), MODE), (dict(T=-1), SHAPE), (dict(E=0), SHAPE), (dict(E=1025, ld=1025), SHAPE),
                   (dict(top=0), SHAPE), (dict(top=33), SHAPE), (dict(E=4, top=5), SHAPE), (dict(ld=63), SHAPE),
                   (dict(x=FAKE + 1), ALIGN), (dict(t=0, x=FAKE + 2), ALIGN), (dict(ids=FAKE + 2), ALIGN),
                   (dict(w=FAKE + 2), ALIGN), (dict(T=1 << 30), OVERFLOW)])


def test_topk_grad(L):
    def call(x=FAKE, t=0, T=4, E=64, ld=64, ids=FAKE, dw=FAKE, top=8, renorm=0, dx=FAKE, ldd=64):
        return L.tq_expert_topk_grad(x, t, T, E, ld, ids, dw, top, renorm, dx, ldd, None)
    assert call() == DEVICE and call(T=0, x=None) == OK
    refuses(call, [(dict(x=None), NULL), (dict(ids=None), NULL), (dict(dw=None), NULL), (dict(dx=None), NULL),
                   (dict(t=3), MODE), (dict(renorm=-1), MODE), (dict(top=65), SHAPE), (dict(ldd=60), SHAPE),
                   (dict(dx=FAKE + 2), ALIGN), (dict(dw=FAKE + 2), ALIGN), (dict(T=1 << 40), OVERFLOW)])


def test_sort(L):
    def call(ids=FAKE, T=4, top=8, E=64, off=FAKE, token=FAKE, place=FAKE):
        return L.tq_expert_sort(ids, T, top, E, off, token, place, None)
    assert call() == DEVICE and call(T=0, ids=None, token=None, place=None) == DEVICE and call(E=4) == DEVICE
    refuses(call, [(dict(ids=None), NULL), (dict(off=None), NULL), (dict(token=None), NULL), (dict(place=None), NULL),
                   (dict(T=-1), SHAPE), (dict(top=0), SHAPE), (dict(top=33), SHAPE), (dict(E=0), SHAPE),
                   (dict(E=1025), SHAPE), (dict(T=1 << 29), OVERFLOW), (dict(ids=FAKE + 2), ALIGN),
                   (dict(off=FAKE + 2), ALIGN), (dict(token=FAKE + 2), ALIGN), (dict(place=FAKE + 2), ALIGN)])


def test_gather(L):
    def call(X=FAKE, t=1, R=4, W=64, ldx=64, rows=FAKE, M=8, Y=FAKE, ldy=64):
        return L.tq_expert_gather(X, t, R, W, ldx, rows, M, Y, ldy, None)
    assert call() == DEVICE and call(M=0, Y=None) == OK and call(R=0, X=None) == DEVICE and call(t=0, W=4) == DEVICE
    refuses(call, [(dict(X=None), NULL), (dict(rows=None), NULL), (dict(Y=None), NULL), (dict(t=2), MODE),
                   (dict(W=60), SHAPE), (dict(W=0), SHAPE), (dict(R=-1), SHAPE), (dict(M=-1), SHAPE),
                   (dict(ldx=56), SHAPE), (dict(ldy=56), SHAPE), (dict(ldx=68), ALIGN), (dict(Y=FAKE + 8), ALIGN),
                   (dict(rows=FAKE + 2), ALIGN), (dict(M=1 << 31), OVERFLOW)])


def test_combine(L):
    def call(Y=FAKE, t=1, R=32, W=64, ldy=64, place=FAKE, w=FAKE, T=4, top=8, O=FAKE, ldo=64):
        return L.tq_expert_combine(Y, t, R, W, ldy, place, w, T, top, O, ldo, None)
    assert call() == DEVICE and call(T=0, O=None) == OK and call(w=None) == DEVICE and call(R=0, Y=None) == DEVICE
    refuses(call, [(dict(Y=None), NULL), (dict(place=None), NULL), (dict(O=None), NULL), (dict(t=2), MODE),
                   (dict(top=0), SHAPE), (dict(top=33), SHAPE), (dict(W=4), SHAPE), (dict(ldo=56), SHAPE),
                   (dict(O=FAKE + 4), ALIGN), (dict(ldy=66), ALIGN), (dict(w=FAKE + 2), ALIGN),
                   (dict(place=FAKE + 2), ALIGN), (dict(T=1 << 30), OVERFLOW)])


def test_combine_grad(L):
    def call(dO=FAKE, ldo=64, Y=FAKE, t=0, R=32, W=64, ldy=64, place=FAKE, w=FAKE, T=4, top=8, dY=FAKE, lddy=64,
             dw=FAKE):
        return L.tq_expert_combine_grad(dO, ldo, Y, t, R, W, ldy, place, w, T, top, dY, lddy, dw, None)
    assert call() == DEVICE and call(T=0, dO=None) == OK and call(w=None, dw=None, Y=None) == DEVICE
    refuses(call, [(dict(dO=None), NULL), (dict(Y=None), NULL), (dict(place=None), NULL), (dict(dY=None), NULL),
                   (dict(t=2), MODE), (dict(top=0), SHAPE), (dict(ldo=60), SHAPE), (dict(lddy=60), SHAPE),
                   (dict(dY=FAKE + 8), ALIGN), (dict(dw=FAKE + 2), ALIGN), (dict(R=1 << 31), OVERFLOW)])
