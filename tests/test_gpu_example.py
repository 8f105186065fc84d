"""The attention layer put together from the library's operators."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("shape", [dict(), dict(width=512, heads=4, heads_kv=4, dim=64, lengths=(5, 130), page=32),
                                   dict(width=512, heads=8, heads_kv=1, dim=256, lengths=(257, 1, 64), page=64)])
def test_attention_layer_follows_fp32(tq, shape):
    """4-bit rounding of keys and values leaves about 0.1 of a row (a step of
    amax / 7, amax about 2.7 sigma, over sqrt(12)), less over many positions; the
    8-bit products below 0.02.  0.2 is beyond them, and far below what a wrong
    position, page or head leaves (about 1).  A graph's step is the same step."""
    from decoder_attention import run
    (prompts, decoded), differ, _ = run(**shape)
    assert prompts <= 0.2 and decoded <= 0.2
    assert differ == 0.0
