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
