"""Tensors that a call makes itself belong to the call's stream (no GPU).

With ``stream`` given, an output made on the current stream could be one that an
earlier kernel there still uses, and zeros filled in there could wipe what the call's
kernel wrote: nothing orders the two streams, and the caller cannot, as both happen
inside the call."""
import contextlib

import pytest

from test_binding_expert import Fake, on0, tq  # noqa: F401


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

    class Made(Fake):
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
