"""The binding's own checks of the 8-bit floating-point products and the experts' calls
(no GPU): tensors that are not what a call needs are refused before the library is
reached."""
import pytest


@pytest.fixture
def tq():
    from dit_convrot_linear_gb300 import build, tq as binding
    build.build()
    import torch
    if torch.cuda.is_available():
        pytest.skip("tensors of the host stand for wrong ones: run where no GPU is visible")
    binding._module()
    return binding


def refused(f, *a, **kw):
    with pytest.raises(ValueError):
        f(*a, **kw)


class Fake:
    """A tensor's description without its memory, on device 0."""

    def __init__(self, shape, dtype, strides=None, device=0):
        import torch
        t = torch.empty(0, dtype=dtype)
        self.shape, self.dtype, self._device, self.device = torch.Size(shape), dtype, device, f"cuda:{device}"
        n = 1
        dense = []
        for s in reversed(shape):
            dense.insert(0, n)
            n *= s
        self._n, self._strides, self._size = n, tuple(strides or dense), t.element_size()
        self._dense = tuple(dense) == self._strides

    def get_device(self):
        return self._device

    def stride(self, i=None):
        return self._strides if i is None else self._strides[i]

    def numel(self):
        return self._n

    def dim(self):
        return len(self.shape)

    def element_size(self):
        return self._size

    def is_contiguous(self):
        return self._dense

    def data_ptr(self):
        return 0x10000


@pytest.fixture
def on0(tq, monkeypatch):
    import torch
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0, raising=False)
    return tq


def reaches(tq, f, *a, **kw):
    """The call passes the binding's checks (and the library finds no device)."""
    with pytest.raises(tq.TQError) as e:
        f(*a, **kw)
    assert e.value.status == 10, e.value


def test_tensors_of_the_host_are_refused(on0):
    import torch
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    refused(on0.quant_act_f8, x)
    refused(on0.expert_sort, torch.zeros(4, 2, dtype=torch.int32), 3)
    refused(on0.expert_topk, torch.zeros(4, 8), 2)


def test_quant(on0):
    import torch
    bf, f32, u8, i32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32
    X, Xq, sx = Fake((4, 896), bf), Fake((4, 896), u8), Fake((7, 4), f32)
    q = on0.quant_act_f8
    reaches(on0, q, X, Xq=Xq, sx=sx)
    reaches(on0, q, Fake((4, 896), bf, (904, 1)), Xq=Xq, sx=sx)
    reaches(on0, q, X, rows=Fake((9,), i32), Xq=Fake((9, 896), u8), sx=Fake((7, 9), f32))
    reaches(on0, q, X, Xq=Fake((4, 896), torch.float8_e4m3fn), sx=sx)
    refused(q, Fake((4, 896), f32), Xq=Xq, sx=sx)
    refused(q, Fake((4, 896), bf, device=1), Xq=Xq, sx=sx)
    refused(q, Fake((896, 4), bf, (1, 896)), Xq=Fake((896, 4), u8), sx=Fake((1, 896), f32))
    refused(q, X, Xq=Fake((4, 880), u8), sx=sx)
    refused(q, X, Xq=Fake((4, 896), u8, (904, 1)), sx=sx)
    refused(q, X, Xq=Xq, sx=Fake((4, 7), f32))
    refused(q, X, Xq=Xq, sx=Fake((7, 4), bf))
    refused(q, X, rows=Fake((4,), torch.int64), Xq=Xq, sx=sx)
    s = on0.swiglu_quant_act_f8
    reaches(on0, s, X, X, Xq=Xq, sx=sx)
    refused(s, X, Fake((4, 880), bf), Xq=Xq, sx=sx)


def test_products(on0):
    import torch
    bf, f32, u8, i32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32
    good = dict(Xq=Fake((4, 896), u8), sx=Fake((7, 4), f32), Wq=Fake((300, 896), u8), sw=Fake((3, 7), f32),
                workspace=Fake((1 << 28,), u8), Y=Fake((4, 300), bf))
    reaches(on0, on0.linear_f8, **good)
    reaches(on0, on0.linear_f8, **{**good, "Y": Fake((9, 304), bf)})
    for kw in (dict(Xq=Fake((4, 880), u8)), dict(sx=Fake((7, 5), f32)), dict(Wq=Fake((300, 880), u8)),
               dict(Wq=Fake((300, 896), bf)), dict(sw=Fake((2, 7), f32)), dict(sw=Fake((3, 7), bf)),
               dict(Y=Fake((4, 299), bf)), dict(Y=Fake((3, 300), bf)), dict(Y=Fake((4, 300), f32)), dict(out="i32"),
               dict(workspace=Fake((1 << 28,), u8, device=1)), dict(workspace=Fake((1 << 28,), torch.int8)),
               dict(Y=Fake((4, 300), bf, (1, 4)))):
        refused(on0.linear_f8, **{**good, **kw})
    good.update(offsets=Fake((6,), i32), Wq=Fake((5, 300, 896), u8), sw=Fake((5, 3, 7), f32))
    reaches(on0, on0.linear_f8_experts, **good)
    for kw in (dict(offsets=Fake((5,), i32)), dict(offsets=Fake((6,), torch.int64)), dict(Wq=Fake((300, 896), u8)),
               dict(sw=Fake((3, 7), f32)), dict(sw=Fake((5, 3, 8), f32))):
        refused(on0.linear_f8_experts, **{**good, **kw})


def test_experts(on0):
    import torch
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    L, ids, w = Fake((6, 40), f32), Fake((6, 4), i32), Fake((6, 4), f32)
    reaches(on0, on0.expert_topk, L, 4, ids=ids, weights=w)
    for kw in (dict(ids=Fake((6, 3), i32)), dict(ids=Fake((6, 4), torch.int64)), dict(weights=Fake((6, 3), f32)),
               dict(weights=Fake((6, 4), bf))):
        refused(on0.expert_topk, L, 4, **{"ids": ids, "weights": w, **kw})
    refused(on0.expert_topk, Fake((6, 40), torch.float16), 4, ids=ids, weights=w)
    reaches(on0, on0.expert_topk_grad, L, ids, w, dlogits=Fake((6, 40), f32))
    refused(on0.expert_topk_grad, L, ids, w, dlogits=Fake((6, 40), bf))
    refused(on0.expert_topk_grad, L, Fake((24,), i32), w, dlogits=L)
    lists = dict(offsets=Fake((41,), i32), token=Fake((24,), i32), place=ids)
    reaches(on0, on0.expert_sort, ids, 40, **lists)
    for kw in (dict(offsets=Fake((40,), i32)), dict(token=Fake((23,), i32)), dict(place=Fake((6, 5), i32))):
        refused(on0.expert_sort, ids, 40, **{**lists, **kw})
    Y, O = Fake((24, 64), bf), Fake((6, 64), bf)
    reaches(on0, on0.expert_combine, Y, ids, w, O=O)
    reaches(on0, on0.expert_combine, Y, ids, O=O)
    for kw in (dict(O=Fake((5, 64), bf)), dict(O=Fake((6, 64), f32)), dict(weights=Fake((6, 3), f32)),
               dict(place=Fake((6, 4), f32))):
        refused(on0.expert_combine, **{"Y": Y, "place": ids, "weights": w, "O": O, **kw})
    reaches(on0, on0.expert_gather, O, Fake((24,), i32), Y=Y)
    refused(on0.expert_gather, O, Fake((24,), i32), Y=Fake((23, 64), bf))
    reaches(on0, on0.expert_combine_grad, O, Y, ids, w, dY=Fake((24, 64), bf), dweights=w)
    refused(on0.expert_combine_grad, Fake((6, 32), bf), Y, ids, w, dY=Y, dweights=w)
    refused(on0.expert_combine_grad, O, Y, ids, w, dY=Y, dweights=Fake((6, 4), bf))


@pytest.mark.parametrize("name", ["int8", "bool", "float8_e5m2"])
def test_other_bytes_are_not_codes(on0, name):
    """A byte of another type would be read as e4m3 and give wrong products quietly."""
    import torch
    bf, f32, u8, i32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32
    other = getattr(torch, name)
    good = dict(Xq=Fake((4, 896), u8), sx=Fake((7, 4), f32), Wq=Fake((300, 896), u8), sw=Fake((3, 7), f32),
                workspace=Fake((1 << 28,), u8), Y=Fake((4, 300), bf))
    refused(on0.linear_f8, **{**good, "Xq": Fake((4, 896), other)})
    refused(on0.linear_f8, **{**good, "Wq": Fake((300, 896), other)})
    refused(on0.quant_act_f8, Fake((4, 896), bf), Xq=Fake((4, 896), other), sx=Fake((7, 4), f32))
    good.update(offsets=Fake((6,), i32), Wq=Fake((5, 300, 896), other), sw=Fake((5, 3, 7), f32))
    refused(on0.linear_f8_experts, **good)


def test_every_call_says_that_the_library_is_missing(on0, monkeypatch):
    """A load that failed is not taken for one that succeeded."""
    import torch

    def missing(*a):
        raise RuntimeError("libtq.so is missing: build it")

    monkeypatch.setattr(on0, "_torch", None)
    monkeypatch.setattr(on0, "_lib", None)
    monkeypatch.setattr(on0, "load", missing)
    for _ in range(3):
        with pytest.raises(RuntimeError, match="is missing"):
            on0.quant_act_f8(Fake((4, 896), torch.bfloat16), Xq=Fake((4, 896), torch.uint8),
                             sx=Fake((7, 4), torch.float32))


def test_a_call_of_another_thread_waits_for_the_library(on0, monkeypatch):
    """While one thread loads, another one does not go past the load."""
    import threading

    import torch
    lib, inside, go = on0._lib, threading.Event(), threading.Event()

    def slow(*a):
        inside.set()
        assert go.wait(20)
        on0._lib = lib
        return lib

    monkeypatch.setattr(on0, "_torch", None)
    monkeypatch.setattr(on0, "_lib", None)
    monkeypatch.setattr(on0, "load", slow)
    out = []

    def call():
        try:
            on0.quant_act_f8(Fake((4, 896), torch.bfloat16), Xq=Fake((4, 896), torch.uint8), sx=Fake((7, 4), torch.float32))
        except Exception as e:
            out.append(e)

    threads = [threading.Thread(target=call) for _ in range(2)]
    threads[0].start()
    assert inside.wait(20)
    threads[1].start()
    threads[1].join(1.0)
    go.set()
    for t in threads:
        t.join(20)
    assert [getattr(e, "status", e) for e in out] == [10, 10]     # both reach the library (which finds no device)


def required():
    """Each call's tensors, all of which it needs."""
    import torch
    bf, f32, u8, i32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32
    X, Xq, sx, ids = Fake((4, 896), bf), Fake((4, 896), u8), Fake((7, 4), f32), Fake((6, 4), i32)
    Y, O, w, L, ws = Fake((24, 64), bf), Fake((6, 64), bf), Fake((6, 4), f32), Fake((6, 40), f32), Fake((1 << 28,), u8)
    made = dict(Xq=Xq, sx=sx)
    product = dict(Xq=Xq, sx=sx, sw=Fake((3, 7), f32), Wq=Fake((300, 896), u8), workspace=ws)
    experts = {**product, "offsets": Fake((6,), i32), "Wq": Fake((5, 300, 896), u8), "sw": Fake((5, 3, 7), f32)}
    # name: tensors that are required, and what the call gets besides
    return {
        "quantize_weights_f8": (dict(W=X), dict(codes=Xq, scales=Fake((1, 7), f32))),
        "quant_act_f8": (dict(X=X), made), "swiglu_quant_act_f8": (dict(G=X, U=X), made),
        "linear_f8": (product, dict(Y=Fake((4, 300), bf))), "linear_f8_experts": (experts, dict(Y=Fake((4, 300), bf))),
        "expert_topk": (dict(logits=L), dict(top=4, ids=ids, weights=w)),
        "expert_topk_grad": (dict(logits=L, ids=ids, dweights=w), dict(dlogits=L)),
        "expert_sort": (dict(ids=ids), dict(experts=40, offsets=Fake((41,), i32), token=Fake((24,), i32), place=ids)),
        "expert_gather": (dict(X=O, rows=Fake((24,), i32)), dict(Y=Y)),
        "expert_combine": (dict(Y=Y, place=ids), dict(O=O)),
        "expert_combine_grad": (dict(dO=O, Y=Y, place=ids), dict(dY=Y, dweights=w)),
    }


@pytest.mark.parametrize("name", sorted(required()))
def test_a_missing_tensor_is_named(on0, name):
    tensors, others = required()[name]
    reaches(on0, getattr(on0, name), **tensors, **others)
    for missing in tensors:
        with pytest.raises(ValueError, match=f"^{missing} is required"):
            getattr(on0, name)(**{**tensors, **others, missing: None})
