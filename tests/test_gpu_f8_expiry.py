"""A bounded wait of the 8-bit floating-point product that runs out.

The test builds a copy of the library whose product expects 16 bytes more of each
stage than its copies bring, with waits of about 1 ms in place of 2 s.  Nothing
traps or spins without a limit: the copies that were issued have landed long before
the CTA leaves.  The status reports the expiry once, nothing is written, and the
library's own product on the same context is right.
"""
import ctypes

import pytest

import f8_ref as ref

pytestmark = pytest.mark.gpu

TIMEOUT = 9


@pytest.fixture(scope="module")
def expiring_lib():
    from dit_convrot_linear_gb300 import build, tq
    path = build.build_variant("f8_expiry", ["TQ_TEST_UNSET_BYTES=16", "TQ_TEST_WAIT_CYCLES=2000000"],
                               ["k_f8_gemm.cu"])
    L = ctypes.CDLL(path)
    for name in ("tq_linear_f8", "tq_linear_f8_experts", "tq_device_status"):
        res, args = tq.SIGNATURES[name]
        fn = getattr(L, name)
        fn.restype, fn.argtypes = res, args
    return L


# few and many tokens
@pytest.mark.parametrize("M", [3, 300])
@pytest.mark.parametrize("experts", [False, True])
def test_expired_wait_is_reported(tq, expiring_lib, M, experts):
    import torch
    N, K, E = 4096, 2048, 2
    g = torch.Generator(device="cuda")
    g.manual_seed(M)
    X = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    W = [tq.quantize_weights_f8((torch.randn(N, K, generator=g, device="cuda") / 45).bfloat16()) for _ in range(E)]
    codes, scales = torch.stack([w[0] for w in W]), torch.stack([w[1] for w in W])
    offsets = torch.tensor([0, M // 3, M], dtype=torch.int32, device="cuda")
    q, sx = tq.quant_act_f8(X)
    work = tq.f8_workspace()
    Y = torch.zeros(M, N, device="cuda")
    assert tq.device_status() == 0
    s = torch.cuda.current_stream().cuda_stream
    L = expiring_lib
    if experts:
        rc = L.tq_linear_f8_experts(q.data_ptr(), sx.data_ptr(), M, K, offsets.data_ptr(), E, codes.data_ptr(),
                                    scales.data_ptr(), N, Y.data_ptr(), 0, N, work.data_ptr(), work.numel(), s)
    else:
        rc = L.tq_linear_f8(q.data_ptr(), sx.data_ptr(), M, K, codes.data_ptr(), scales.data_ptr(), N, Y.data_ptr(), 0,
                            N, work.data_ptr(), work.numel(), s)
    assert rc == 0                                  # launched; the waits run out on the device
    assert L.tq_device_status(s) == TIMEOUT
    assert L.tq_device_status(s) == 0               # reading clears it
    assert torch.all(Y == 0)
    work = tq.f8_workspace()
    ends = [0, M // 3, M] if experts else [0, M]
    if experts:
        Y = tq.linear_f8_experts(q, sx, offsets, codes, scales, work, out="f32")
    else:
        Y = tq.linear_f8(q, sx, codes[0], scales[0], work, out="f32")
    assert tq.device_status() == 0
    for e, (a, b) in enumerate(zip(ends, ends[1:])):
        want, S = ref.product(q[a:b], sx[:, a:b], codes[e], scales[e])
        assert ((Y[a:b].double() - want).abs() <= ref.product_bar(K, S, want, False)).all()
