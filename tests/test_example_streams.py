"""The experts' example warms up on a stream of its own (no GPU): it has to wait for the
stream on which the weights and the rows are made, and that one for it."""
import contextlib
import os
import sys

import pytest

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


class Stream:
    def __init__(self, name="side"):
        self.name = name

    def wait_stream(self, other):
        LOG.append(f"{self.name} waits for {other.name}")


class Captures(Exception):
    """The warm-up is over."""


LOG = []


def test_warm_up_is_ordered_behind_the_current_stream(monkeypatch):
    import expert_ffn
    import torch
    del LOG[:]
    at = [Stream("main")]
    randn = torch.randn

    class Layer:
        def __init__(self, *a):
            LOG.append(f"weights on {at[-1].name}")

        def __call__(self, x, r):
            LOG.append(f"layer on {at[-1].name}")

    @contextlib.contextmanager
    def on(stream):
        at.append(stream)
        yield
        at.pop()

    def graph():
        raise Captures

    generator = torch.Generator
    monkeypatch.setattr(expert_ffn, "Experts", Layer)
    monkeypatch.setattr(torch, "Generator", lambda device=None: generator())
    monkeypatch.setattr(torch, "randn", lambda *s, generator, device: randn(*s, generator=generator))
    for name, v in (("Stream", Stream), ("stream", on), ("current_stream", lambda d=None: at[-1]),
                    ("synchronize", lambda: LOG.append("synchronize")), ("CUDAGraph", graph)):
        monkeypatch.setattr(torch.cuda, name, v)
    with pytest.raises(Captures):
        expert_ffn.run(width=16, tokens=2)
    assert LOG == ["weights on main", "side waits for main", "layer on side", "main waits for side", "synchronize"]
