"""Tensors that a call makes itself belong to the call's stream (no GPU).

With ``stream`` given, an output made on the current stream could be one that an
earlier kernel there still uses, and zeros filled in there could wipe what the call's
kernel wrote: nothing orders the two streams, and the caller cannot, as both happen
inside the call."""
import contextlib
import types

import pytest

from test_binding_expert import Fake, on0, tq  # noqa: F401


class Dense(Fake):
    """With what the other calls ask of a tensor besides."""
    is_cuda = True

    def __init__(self, *a, **kw):
        super().__init__(*a, **kw)
        self.device = types.SimpleNamespace(index=0)


class Stream:
    """A stream's handle."""
    cuda_stream = 0x5


def f8_calls():
    import torch
    bf, f32, u8, i32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32
    X, q, sx, ids = Fake((4, 896), bf), Fake((4, 896), u8), Fake((7, 4), f32), Fake((6, 4), i32)
    Y, w, ws = Fake((24, 64), bf), Fake((6, 4), f32), Fake((1 << 28,), u8)
    return {
        "quantize_weights_f8": ((X,), 2),
        "quant_act_f8": ((X,), 2),
        "swiglu_quant_act_f8": ((X, X), 2),
        "linear_f8": ((q, sx, Fake((300, 896), u8), Fake((3, 7), f32), ws), 1),
        "linear_f8_experts": ((q, sx, Fake((6,), i32), Fake((5, 300, 896), u8), Fake((5, 3, 7), f32), ws), 1),
        "expert_topk": ((Fake((6, 40), f32), 4), 2),
        "expert_topk_grad": ((Fake((6, 40), f32), ids, w), 1),
        "expert_sort": ((ids, 40), 3),
        "expert_gather": ((Fake((6, 64), bf), Fake((24,), i32)), 1),
        "expert_combine": ((Y, ids, w), 1),
        "expert_combine_grad": ((Fake((6, 64), bf), Y, ids, w), 2),
    }


@pytest.fixture
def made(monkeypatch):
    """(stream at the time, tensor) of every tensor that is made, and the stream that
    each records."""
    import torch
    at, log, recorded = ["current"], [], []

    class Made(Dense):
        def record_stream(self, s):
            recorded.append(s)

    def make(shape, dtype=None, device=None):
        t = Made(shape if hasattr(shape, "__len__") else (shape,), dtype)
        log.append((at[-1], t))
        return t

    @contextlib.contextmanager
    def on(stream):
        at.append(stream)
        yield
        at.pop()

    fake = make
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: at[-1])
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle: f"stream {handle}")
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda shape, dtype=None, device=None: (
        empty(shape, dtype=dtype) if device is None else fake(shape, dtype, device)))
    monkeypatch.setattr(torch, "zeros", fake)
    return log, recorded


@pytest.mark.parametrize("name", sorted(f8_calls()))
def test_made_on_the_call_s_stream(on0, made, name):  # noqa: F811
    args, n = f8_calls()[name]
    log, recorded = made
    with pytest.raises(on0.TQError):                   # no device: the checks have passed
        getattr(on0, name)(*args, stream=Stream())
    assert [at for at, _ in log] == ["stream 5"] * n
    assert recorded == ["current"] * n                 # the caller's stream holds it too
    del log[:], recorded[:]
    with pytest.raises(on0.TQError):
        getattr(on0, name)(*args)
    assert [at for at, _ in log] == ["current"] * n and not recorded


def other_calls(tq):  # noqa: F811
    import torch
    bf, f32, u8, i8, i32 = torch.bfloat16, torch.float32, torch.uint8, torch.int8, torch.int32
    big, X, sx, w = Dense((1 << 24,), u8), Dense((4, 896), bf), Dense((4,), f32), Dense((896,), f32)
    sw, heads = Dense((1024,), f32), Dense((4, 2, 128), bf)
    cache = types.SimpleNamespace(pool=big, npages=4, page_size=16, heads=2, dim=128)
    batch = tq.KV4Batch(cache, Dense((4, 1), i32), Dense((4,), i32), Dense((5,), i32), 4)
    return {
        "quantize_weights": (X, 8), "quantize_weights_blocked": (X, 4, 32), "rotate_quant_act": (X,),
        "linear_blocked": (X, big, sw, 128, 8, 128), "rotate_act_bf16": (X,), "linear": (X, big, sw, 128, 8, "W8A8"),
        "linear_swiglu": (X, X, big, sw, 128, 8, "W8A16"), "linear_q8": (Dense((4, 896), i8), sx, big, sw, 128, 8),
        "rotate_quant_act_tiled": (X,), "modnorm_quant_act_tiled": (X, w, w), "swiglu_quant_act_tiled": (X, X),
        "linear_tiled": (big, sx, 4, 896, big, sw, 128, 8), "tile_weights": (big, 128, 896, 8),
        "linear_tt": (big, sx, 4, 896, big, sw, 128, 8), "linear_tt_ex": (big, sx, 4, 896, big, sw, 128, 8),
        "rmsnorm_quant_act": (X, w), "rmsnorm": (X, w), "rmsnorm_quant_act_tiled": (X, w),
        "rope": (heads, Dense((1, 4), i32), tq.RopeSpec(Dense((64,), f32))), "kv4_read": (batch,),
        "kv4_attention": (batch, heads, 0.1, big),
    }


OTHERS = {"quantize_weights": 2, "quantize_weights_blocked": 2, "rotate_quant_act": 2, "linear_blocked": 1,
          "rotate_act_bf16": 1, "linear": 2, "linear_swiglu": 1, "linear_q8": 1, "rotate_quant_act_tiled": 2,
          "modnorm_quant_act_tiled": 2, "swiglu_quant_act_tiled": 2, "linear_tiled": 1, "tile_weights": 1,
          "linear_tt": 1, "linear_tt_ex": 1, "rmsnorm_quant_act": 2, "rmsnorm": 1, "rmsnorm_quant_act_tiled": 2,
          "rope": 1, "kv4_read": 2, "kv4_attention": 1}


@pytest.mark.parametrize("name", sorted(OTHERS))
def test_other_calls_tensors_are_made_there_too(on0, made, name, monkeypatch):  # noqa: F811
    log, recorded = made
    monkeypatch.setattr(on0, "linear_workspace_bytes", lambda *a: 4096)      # as a device's would be
    args = other_calls(on0)[name]
    with pytest.raises(on0.TQError):
        getattr(on0, name)(*args, stream=Stream())
    assert [at for at, _ in log] == ["stream 5"] * OTHERS[name]
    assert recorded == ["current"] * OTHERS[name]


@pytest.mark.parametrize("capturing", [False, True])
@pytest.mark.parametrize("name", ["f8_workspace", "kv4_workspace", "split_workspace"])
def test_a_workspace_is_zeroed_on_return(on0, monkeypatch, name, capturing):  # noqa: F811
    """Its first use may be on any stream: the fill is over when the call returns (a
    capture's is a node of the graph and cannot be waited for)."""
    import torch
    log = []

    def zeros(shape, dtype=None, device=None):
        log.append(("zeros", device))
        return Dense((shape,), dtype)

    stream = types.SimpleNamespace(synchronize=lambda: log.append("synchronize"))
    monkeypatch.setattr(torch, "zeros", zeros)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: stream)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing)
    assert getattr(on0, name)().dtype is torch.uint8
    assert log == [("zeros", "cuda")] + ([] if capturing else ["synchronize"])
