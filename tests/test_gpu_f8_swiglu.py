"""The SwiGLU operand's codes against the range that its arithmetic allows.

h = g / (1 + e^-g) * u is formed in fp32 with the hardware's exponential and division.
By their published bounds (CUDA C++ programming guide, intrinsic functions) __expf(x)
is off by 2 + floor(|1.173 x|) units in the last place and __fdividef by 2 where the
divisor lies within 2^+-126; the sum and the product by u round by half a unit each.  A
unit is at most 2^-23 of a value, and an error of e^-g reaches 1 + e^-g at most in
full.  So for |g| <= 87

    |h' - h| <= (5 + 1.173 |g|) 2^-23 |h|   (1.001 of it, for the products of errors),

and by at most 2^-148 more where something is subnormal.  Below -87 h' may be zero.  A code
is one rounding of h' / s: it lies between the codes of the two ends of that range, and
the scale is that of a largest value within it.
"""
import pytest

import f8_ref as ref

pytestmark = pytest.mark.gpu


def operands(kind, M, K):
    import torch
    g = torch.Generator(device="cuda").manual_seed(M + K)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    if kind == "ordinary":
        both = 3.0 * n(M, 2 * K)
        return both[:, :K].bfloat16(), both[:, K:].bfloat16()
    G = 180.0 * torch.rand(M, K, generator=g, device="cuda") - 90.0
    if kind == "wide":                                  # gates of all sizes beside each other
        return G.bfloat16(), n(M, K).bfloat16()
    # blocks of very negative gates, brought back to ordinary sizes by the other half
    G = -(87.0 * torch.rand(M, -(-K // 128), generator=g, device="cuda")).repeat_interleave(128, 1)[:, :K]
    G = (G + 0.3 * n(M, K)).clamp(max=-1e-3).bfloat16()
    return G, (n(M, K) * torch.exp(-G.float())).bfloat16()


@pytest.mark.parametrize("kind", ["ordinary", "wide", "negative"])
@pytest.mark.parametrize("M,K", [(1, 16), (33, 1024), (6, 2000), (64, 4096)])
def test_codes_within_the_arithmetic_s_range(tq, kind, M, K):
    import torch
    G, U = operands(kind, M, K)
    q, s = tq.swiglu_quant_act_f8(G, U)
    g, u = G.double().cpu(), U.double().cpu()
    h = g / (1.0 + torch.exp(-g)) * u
    near = h.abs() * torch.where(g < -87.0, 1.0, (5.0 + 1.173 * g.abs()) * 2.0 ** -23 * 1.001) + 2.0 ** -148
    s = s.cpu().double().t()
    for i in range(M):
        for j in range(s.shape[1]):
            at = slice(128 * j, 128 * j + 128)
            low = float((h[i, at].abs() - near[i, at]).clamp(min=0.0).max())
            high = float((h[i, at].abs() + near[i, at]).max())
            assert ref.power_scale(low) <= float(s[i, j]) <= ref.power_scale(high), (i, j)
    wide = s.repeat_interleave(128, 1)[:, :K]
    v = ref.decode(q.cpu())
    assert (v[wide == 0.0] == 0.0).all()
    some = wide > 0.0
    x, d, wide = h[some], near[some], wide[some]
    low = ref.decode(ref.encode(((x - d) / wide).clamp(-ref.MOST, ref.MOST)))
    high = ref.decode(ref.encode(((x + d) / wide).clamp(-ref.MOST, ref.MOST)))
    assert ((low <= v[some]) & (v[some] <= high)).all()
    assert tq.device_status() == 0
