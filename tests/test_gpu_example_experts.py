"""The experts' layer put together from the library's operators."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("shape", [dict(), dict(width=256, hidden=144, experts=3, top=3, tokens=1),
                                   dict(width=512, hidden=128, experts=64, top=8, tokens=700)])
def test_layer_follows_fp32(tq, shape):
    """Four operands rounded to e4m3, 2^-4 of a value at most (0.03 at random), and
    bf16's 2^-8: about 0.07 of the output; a wrong row or expert leaves about 1.  A graph's
    step is the same step."""
    from expert_ffn import run
    err, differ, _ = run(**shape)
    assert err <= 0.1
    assert differ == 0.0


def test_way_back(tq):
    """The gradients of the rows and of the logits, by the formula of the library's own
    forward (64-bit autograd of the choice's softmax and the sum)."""
    import torch
    from expert_ffn import Experts
    layer = Experts(256, 128, 12, 3)
    g = torch.Generator(device="cuda").manual_seed(3)
    x, r, dO = (torch.randn(37, 256, generator=g, device="cuda").bfloat16() for _ in range(3))
    layer(x, r)
    dy, dlogits = layer.backward(dO)
    _, logits, ids, _, place, y = layer.saved
    lo, rows = logits.double().requires_grad_(), y.double().requires_grad_()
    w = torch.softmax(torch.gather(lo, 1, ids.long()), 1)
    (w[..., None] * rows[place.long()]).sum(1).backward(dO.double())
    # dy: w within 2^-20 of itself, rounded to bf16; dlogits: dot products of 256 terms in
    # fp32 (2^-24 each, of the sum of magnitudes), then w (dw - sum w dw)
    assert ((dy.double() - rows.grad).abs() <= rows.grad.abs() * (2.0 ** -8 + 2.0 ** -19)).all()
    size = (dO.double().abs()[:, None] * y.double().abs()[place.long()]).sum(-1).max(1, keepdim=True).values
    assert ((dlogits.double() - lo.grad).abs() <= size * (256 * 2.0 ** -24 + 2.0 ** -19)).all()
    assert tq.device_status() == 0
