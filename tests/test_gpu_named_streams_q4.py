"""The 4-bit calls on a named stream while another one is current: what they
make (outputs, workspaces) is made and cleared on the stream they run on."""
import pytest
import torch

import bit_gemv_q4_b200 as gq
from test_gpu_named_streams import same

pytestmark = pytest.mark.gpu

M, K = 256, 2048


def calls():
    g = torch.Generator().manual_seed(3)
    w = torch.randn(M * K, generator=g).cuda()
    x = torch.randn(1, K, generator=g).half().cuda()
    X = torch.randn(40, K, generator=g).bfloat16().cuda()
    q, k = gq.gq_quantize_q4_0(w), gq.gq_quantize_ksb(w)
    t = gq.gq_repack(gq.GQ_FMT_Q4_0, q, M, K)
    return {
        "quantize": lambda **kw: [gq.gq_quantize_q4_0(w, **kw), gq.gq_quantize_ksb(w, **kw)],
        "quantize, reference rule": lambda **kw: [gq.gq_quantize_q4_0_ex(w, gq.GQ_QUANT_REF_RULE, **kw)],
        "dequantize": lambda **kw: [gq.gq_dequantize_q4_0(q, M * K, **kw), gq.gq_dequantize_ksb(k, M * K, **kw)],
        "gemv": lambda **kw: [gq.gq_gemv_q4_0(q, M, K, x, **kw), gq.gq_gemv_ksb(k, M, K, x, **kw)],
        "gemv with a workspace": lambda **kw: [gq.gq_gemv_q4_0(q, M, K, x, workspace="auto", **kw)],
        "grouped gemv": lambda **kw: gq.gq_gemv_q4_0_grouped([q, q], [M, M], K, x, **kw),
        "gemm": lambda **kw: [gq.gq_gemm_q4_0(q, M, K, X, **kw), gq.gq_gemm_ksb(k, M, K, X, **kw)],
        "gemv without allocation": lambda **kw: [gq.gq_gemv_q4_0_noalloc(q, M, K, x, **kw)],
        "read": lambda **kw: [gq.gq_stream_read(q, **kw)],
        "repack": lambda **kw: [gq.gq_repack(gq.GQ_FMT_KSB, k, M, K, **kw)],
        "tiled gemv": lambda **kw: [gq.gq_gemv_q4_0_tiled(t, M, K, x, **kw)],
        "grouped tiled gemv": lambda **kw: gq.gq_gemv_q4_0_tiled_grouped([t, t], [M, M], K, x, **kw),
    }


NAMES = ["quantize", "quantize, reference rule", "dequantize", "gemv", "gemv with a workspace", "grouped gemv",
         "gemm", "gemv without allocation", "read", "repack", "tiled gemv", "grouped tiled gemv"]


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("named", ["a stream", "a raw handle", "the default stream", "handle 0"])
def test_outputs_and_workspaces_are_made_on_the_named_stream(name, named, monkeypatch):
    call = calls()[name]
    want = call()
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    stream = {"a stream": side, "a raw handle": side.cuda_stream, "the default stream": torch.cuda.default_stream(),
              "handle 0": 0}[named]
    on = side.cuda_stream if "default" not in named and named != "handle 0" else 0
    monkeypatch.setattr(gq, "_gemv_ws", {})
    seen = []

    def watched(make):
        def made(*args, **kw):
            seen.append(torch.cuda.current_stream().cuda_stream)
            return make(*args, **kw)
        return made

    monkeypatch.setattr(torch, "empty", watched(torch.empty))
    monkeypatch.setattr(torch, "zeros", watched(torch.zeros))
    with torch.cuda.stream(other):
        got = call(stream=stream)
    torch.cuda.synchronize()
    assert seen and all(s == on for s in seen)
    assert same(got, want)
