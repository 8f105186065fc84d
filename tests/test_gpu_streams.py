"""Calls on a stream of their own (``stream=``) while the current stream is busy, with
outputs that the call makes: complete on that stream, and not touched by the other one
later.  Bit for bit what the same call gives without ``stream``."""
import pytest

pytestmark = pytest.mark.gpu

BUSY = 200_000_000            # cycles: 0.1 s


def calls(tq):
    import torch
    g = torch.Generator(device="cuda").manual_seed(3)
    M, K, N, E, top = 200, 896, 300, 6, 2
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, both = n(M, K).bfloat16(), n(M, 2 * K).bfloat16()
    W = n(E, N, K).bfloat16()
    q, sx = tq.quant_act_f8(x)
    Wq, sw = tq.quantize_weights_f8(W)
    logits, dw = n(M // top, E), n(M // top, top)
    ids, w = tq.expert_topk(logits, top)
    ids[::5, 1] = -1                                   # rows of no expert: left as the call's zeros
    offsets, token, place = tq.expert_sort(ids, E)
    y, do, ws = n(M, 64).bfloat16(), n(M // top, 64).bfloat16(), tq.f8_workspace()
    codes, s8 = tq.quantize_weights(W[0], 8)
    gamma, qkv = n(K).abs(), n(40, 2, 128).bfloat16()
    cache = tq.KV4Cache(8, 16, 2, 128)
    i32 = dict(dtype=torch.int32, device="cuda")
    batch = tq.KV4Batch(cache, torch.arange(8, **i32).view(2, 4), torch.tensor([30, 10], **i32),
                        torch.tensor([0, 30, 40], **i32), 40, 30)
    tq.kv4_append(batch, qkv, qkv.flip(0).contiguous())
    kws = tq.kv4_workspace()
    return {
        "linear": lambda **s: tq.linear(x, codes, s8, N, 8, "W8A8", **s),
        "rmsnorm_quant_act": lambda **s: tq.rmsnorm_quant_act(x, gamma, **s),
        "kv4_read": lambda **s: tq.kv4_read(batch, **s),
        "kv4_attention": lambda **s: tq.kv4_attention(batch, qkv, 128 ** -0.5, kws, **s),
        "quantize_weights_f8": lambda **s: tq.quantize_weights_f8(W, **s),
        "quant_act_f8": lambda **s: tq.quant_act_f8(x, **s),
        "swiglu_quant_act_f8": lambda **s: tq.swiglu_quant_act_f8(both[:, :K], both[:, K:], **s),
        "linear_f8": lambda **s: tq.linear_f8(q, sx, Wq[0], sw[0], ws, **s),
        "linear_f8_experts": lambda **s: tq.linear_f8_experts(q, sx, offsets, Wq, sw, ws, **s),
        "expert_topk": lambda **s: tq.expert_topk(logits, top, **s),
        "expert_topk_grad": lambda **s: tq.expert_topk_grad(logits, ids, dw, **s),
        "expert_sort": lambda **s: tq.expert_sort(ids, E, **s),
        "expert_gather": lambda **s: tq.expert_gather(do, token, **s),
        "expert_combine": lambda **s: tq.expert_combine(y, place, w, **s),
        "expert_combine_grad": lambda **s: tq.expert_combine_grad(do, y, place, w, **s),
    }


NAMES = ["quantize_weights_f8", "quant_act_f8", "swiglu_quant_act_f8", "linear_f8", "linear_f8_experts", "expert_topk",
         "expert_topk_grad", "expert_sort", "expert_gather", "expert_combine", "expert_combine_grad",
         "linear", "rmsnorm_quant_act", "kv4_read", "kv4_attention"]


def several(v):
    return v if isinstance(v, tuple) else (v,)


@pytest.mark.parametrize("name", NAMES)
def test_outputs_made_while_the_current_stream_is_busy(tq, name):
    import torch
    f = calls(tq)[name]
    want = several(f())
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    # once with nothing in the way (kernels are loaded, each stream has its memory), once busy
    for cycles in (0, BUSY):
        if cycles:
            torch.cuda._sleep(cycles)
        got = several(f(stream=side))
        with torch.cuda.stream(side):                  # (waits for the side stream alone)
            same = [torch.equal(a, b) for a, b in zip(got, want)]
        busy = not torch.cuda.current_stream().query()
        torch.cuda.synchronize()
        assert all(same) and all(torch.equal(a, b) for a, b in zip(got, want))
    assert busy                                        # the other stream was not waited for
    assert tq.device_status() == 0


@pytest.mark.parametrize("name", ["f8_workspace", "kv4_workspace", "split_workspace"])
def test_a_workspace_may_be_used_on_any_stream_at_once(tq, name):
    """Zeros on another stream that waits for nothing, in memory that held something else,
    while the stream that fills it is busy."""
    import torch
    side = torch.cuda.Stream()
    old = getattr(tq, name)().fill_(255)
    size = old.numel()
    with torch.cuda.stream(side):                      # (the side stream has its memory)
        assert int(old.count_nonzero()) == size
    torch.cuda.synchronize()
    del old
    torch.cuda._sleep(BUSY)
    ws = getattr(tq, name)()
    with torch.cuda.stream(side):
        assert int(ws.count_nonzero()) == 0
    torch.cuda.synchronize()
    assert ws.numel() == size and int(ws.count_nonzero()) == 0


def test_a_workspace_made_in_a_capture(tq):
    """A workspace that a graph makes itself is filled by the graph at every replay."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(24, 2048, generator=g, device="cuda").bfloat16()
    W = tq.quantize_weights_f8(torch.randn(896, 2048, generator=g, device="cuda").bfloat16())
    want = tq.linear_f8(*tq.quant_act_f8(x), *W, tq.f8_workspace())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Y = tq.linear_f8(*tq.quant_act_f8(x), *W, tq.f8_workspace())
    for _ in range(3):
        Y.zero_()
        graph.replay()
        assert torch.equal(Y, want)
    assert tq.device_status() == 0


def test_no_tokens_on_a_stream(tq):
    """Outputs without memory have nothing to record."""
    import torch
    side = torch.cuda.Stream()
    x = torch.empty(0, 128, dtype=torch.bfloat16, device="cuda")
    q, sx = tq.quant_act_f8(x, stream=side)
    off, token, place = tq.expert_sort(torch.empty(0, 2, dtype=torch.int32, device="cuda"), 3, stream=side)
    assert q.shape == (0, 128) and sx.shape == (1, 0) and token.shape == (0,) and place.shape == (0, 2)
    assert tq.expert_gather(x, token, stream=side).shape == (0, 128)
    side.synchronize()
    assert off.tolist() == [0, 0, 0, 0]
    assert tq.device_status() == 0


def test_a_stream_within_a_capture(tq):
    """A graph with a branch on a stream of its own, whose outputs the calls make."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(9)
    x = torch.randn(70, 512, generator=g, device="cuda").bfloat16()
    W = tq.quantize_weights_f8(torch.randn(256, 512, generator=g, device="cuda").bfloat16())
    ws, side = tq.f8_workspace(), torch.cuda.Stream()
    want = tq.linear_f8(*tq.quant_act_f8(x), *W, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        Y = tq.linear_f8(*tq.quant_act_f8(x, stream=side), *W, ws, stream=side)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        Y.zero_()
        graph.replay()
        assert torch.equal(Y, want)
    assert tq.device_status() == 0
