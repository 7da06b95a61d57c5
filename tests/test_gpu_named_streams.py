"""Calls on a named stream that make their own outputs, while another stream is
the current one: the memory has to be the named stream's, not memory that the
current stream freed and may still be reading."""
import pytest
import torch

import bit_gemv_q4_b200 as gq
from gpu_helpers import Q40
from test_gpu_moe import Layer, inputs

pytestmark = pytest.mark.gpu


def calls():
    m = Layer(Q40, 8, 512, 192)
    x, ids, w = inputs(5, 512, 8, 3, "f16", seed=4)
    Wr = torch.randn(8, 512, device="cuda")
    W, ws = gq.gq_quantize_fp8(torch.randn(300, 512, device="cuda"), 128)
    X = torch.randn(40, 512, device="cuda")
    q, s = gq.gq_quantize_fp8(X, 1)
    return {
        "route": lambda **kw: gq.gq_moe_route(x, Wr, 3, **kw),
        "layer": lambda **kw: (m(x, ids, w, **kw),),
        "quantize": lambda **kw: gq.gq_quantize_fp8(X, 1, **kw),
        "dequantize": lambda **kw: (gq.gq_dequantize_fp8(q, s, 1, **kw),),
        "product": lambda **kw: (gq.gq_gemm_fp8(W, ws, q, s, **kw),),
        "product of one token": lambda **kw: (gq.gq_gemm_fp8(W, ws, q[:1], s[:1], **kw),),
    }


NAMES = ["route", "layer", "quantize", "dequantize", "product", "product of one token"]


def same(a, b):
    return all(torch.equal(p.view(torch.uint8), r.view(torch.uint8)) for p, r in zip(a, b))


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("raw", [False, True])
def test_memory_that_the_current_stream_still_reads_is_left_alone(name, raw):
    call = calls()[name]
    want = call()
    side = torch.cuda.Stream()
    stream = side.cuda_stream if raw else side
    torch.cuda.synchronize()
    call(stream=stream)  # its workspace is made
    torch.cuda.synchronize()
    # tensors of the outputs' sizes that the current stream reads late and whose memory is free before
    old = [torch.full((o.numel() * o.element_size(),), 0x5A, dtype=torch.uint8, device="cuda") for o in want]
    kept = [torch.empty_like(o) for o in old]
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)  # cycles, about 50 ms
    for a, b in zip(old, kept):
        b.copy_(a)
    del old, a
    got = call(stream=stream)
    side.synchronize()
    assert same(got, want)
    torch.cuda.synchronize()
    assert all(bool((b == 0x5A).all()) for b in kept)
    assert same(got, want)


@pytest.mark.parametrize("name", NAMES)
def test_named_stream_inside_a_capture(name):
    call = calls()[name]
    want = call()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = call(stream=side)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(2):
        for o in got:
            o.view(torch.uint8).zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert same(got, want)


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("stream", [0, 1, "object"])
def test_the_default_stream_named_while_another_is_current(name, stream, monkeypatch):
    # its workspace and its outputs are made, and the workspace cleared, on the default stream
    call = calls()[name]
    want = call()
    torch.cuda.synchronize()
    monkeypatch.setattr(gq, "_call_ws", {})
    seen = []

    def watched(make):
        def made(*args, **kw):
            seen.append(torch.cuda.current_stream().cuda_stream)
            return make(*args, **kw)
        return made

    monkeypatch.setattr(torch, "zeros", watched(torch.zeros))
    monkeypatch.setattr(torch.Tensor, "new_empty", watched(torch.Tensor.new_empty))
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = call(stream=torch.cuda.default_stream() if stream == "object" else stream)
    torch.cuda.synchronize()
    assert same(got, want)
    assert seen and all(s == 0 for s in seen)
