"""The binding's own part of the attention layer's calls, without a GPU: the
tensors are stand-ins that hold a shape, strides and an address."""
import types

import pytest


@pytest.fixture
def binding():
    from dit_convrot_linear_gb300 import tq
    return tq


class Stub:
    """What the binding asks of a CUDA tensor."""
    is_cuda = True

    def __init__(self, dtype, shape, strides=None, at=0x10000):
        import torch
        self._t = torch.empty(0, dtype=dtype)
        self.dtype, self.shape, self.at = dtype, tuple(shape), at
        dense = []
        for n in reversed(shape):
            dense.insert(0, dense[0] * inner if dense else 1)
            inner = n
        self._strides = tuple(dense) if strides is None else tuple(strides)
        self.dense = self._strides == tuple(dense)

    def dim(self):
        return len(self.shape)

    def stride(self, i=None):
        return self._strides if i is None else self._strides[i]

    def numel(self):
        n = 1
        for k in self.shape:
            n *= k
        return n

    def element_size(self):
        return self._t.element_size()

    def is_contiguous(self):
        return self.dense

    def data_ptr(self):
        return self.at


def batch(tq, shape, strides, q_start=None):
    import torch
    cache = types.SimpleNamespace(pool=Stub(torch.uint8, (1 << 20,)), npages=64, page_size=16, heads=2, dim=128)
    n = shape[0]
    return tq.KV4Batch(cache, Stub(torch.int32, shape, strides), Stub(torch.int32, (n,)), Stub(torch.int32, (n + 1,)), n)


@pytest.mark.parametrize("strides", [(0, 1), (1, 1), (7, 1)])
def test_page_table_whose_rows_overlap_is_refused(binding, strides):
    """One row of pages shared by all sequences (an expanded tensor), and rows
    closer than they are long: the kernels would read past the tensor."""
    with pytest.raises(ValueError, match="table"):
        batch(binding, (4, 8), strides)


@pytest.mark.parametrize("shape,strides,ldt", [((4, 8), (8, 1), 8), ((4, 8), (12, 1), 12), ((1, 8), (0, 1), 8),
                                               ((1, 8), (3, 1), 8), ((1, 8), (40, 1), 40), ((3, 1), (1, 1), 1)])
def test_page_table_row_step(binding, shape, strides, ldt):
    """The step between rows as it is; one row has none, its length stands for it."""
    assert batch(binding, shape, strides)._c.ldt == ldt


def test_two_threads_share_a_rope_spec(binding, monkeypatch):
    """A model's spec serves calls from several threads: each call's positions
    are its own, whatever another call does between its set-up and its launch."""
    import threading

    import torch
    spec = binding.RopeSpec(Stub(torch.float32, (64,), at=0x500), axis=[0, 1] * 32)
    before = bytes(spec._c)
    both, seen, wrong = threading.Barrier(2, timeout=20), {}, []

    def tq_rope(x, tokens, heads, dim, ldx, c, y, ldy, stream):
        both.wait()                          # both calls are set up
        s = binding.RopeSpecC.from_address(c)
        seen[x] = (s.pos, s.naxes, s.ldpos, s.inv_freq, s.pairs, bytes((binding.ctypes.c_uint8 * 64).from_address(s.axis)))
        both.wait()
        return 0

    monkeypatch.setattr(binding, "_lib", types.SimpleNamespace(tq_rope=tq_rope))
    stream = types.SimpleNamespace(cuda_stream=0)

    def call(x, pos, axes, tokens):
        try:
            X = Stub(torch.bfloat16, (tokens, 2, 128), at=x)
            binding.rope(X, Stub(torch.int32, (axes, tokens), at=pos), spec, Y=X, stream=stream)
        except Exception as e:               # noqa: BLE001  (for the main thread to show)
            wrong.append(e)

    threads = [threading.Thread(target=call, args=a) for a in ((0x1000, 0x2000, 2, 5), (0x3000, 0x4000, 4, 9))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong
    axis = bytes([0, 1] * 32)
    assert seen == {0x1000: (0x2000, 2, 5, 0x500, 64, axis), 0x3000: (0x4000, 4, 9, 0x500, 64, axis)}
    assert bytes(spec._c) == before          # a call leaves the spec as it is
