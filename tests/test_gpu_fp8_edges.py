"""8-bit blocks at the edges: K below one group of 128 through the tensor-core
product, and bytes around the outputs of the quantizer, the decoder and the
router, which have to stay what they were."""
import pytest
import torch

import bit_gemv_q4_b200 as gq
from test_gpu_fp8 import DT, check, operands

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,K,B", [
    (200, 16, 40), (200, 48, 17), (129, 112, 130), (300, 16, 1000),      # 128 x 128 tiles
    (6000, 48, 1500), (9000, 112, 2500),                                  # pairs, 256 x 256
])
@pytest.mark.parametrize("yt", ["f32", "bf16"])
def test_gemm_of_less_than_a_group(M, K, B, yt):
    W, ws, X, xs = operands(M, K, B, M + K + B)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    Y = gq.gq_gemm_fp8(W, ws, X, xs, y_dtype=DT[yt], dev_status=st)
    check(Y, W, ws, X, xs)
    assert int(st.item()) == 0


GUARD = 1024  # bytes on either side


def guarded(shape, dtype):
    """(a tensor of `shape` inside a buffer of bytes 0xA5, a call that looks at the rest of them)"""
    n = torch.Size(shape).numel() * torch.empty(0, dtype=dtype).element_size()
    buf = torch.full((n + 2 * GUARD,), 0xA5, dtype=torch.uint8, device="cuda")

    def intact():
        return bool((buf[:GUARD] == 0xA5).all()) and bool((buf[GUARD + n:] == 0xA5).all())
    return buf[GUARD:GUARD + n].view(dtype).view(shape), intact


@pytest.mark.parametrize("R,K", [(1, 16), (3, 144), (7, 4096), (129, 400), (300, 1040), (128, 128)])
@pytest.mark.parametrize("rows", [1, 128])
def test_bytes_around_quantizer_and_decoder_outputs(R, K, rows):
    x = torch.randn(R, K, device="cuda", generator=torch.Generator("cuda").manual_seed(R + K))
    q, around_q = guarded((R, K), torch.float8_e4m3fn)
    s, around_s = guarded((-(-R // rows), -(-K // 128)), torch.float32)
    gq.gq_quantize_fp8(x, rows, out=q, scales=s)
    want_q, want_s = gq.gq_quantize_fp8(x, rows)
    assert torch.equal(q.view(torch.uint8), want_q.view(torch.uint8)) and torch.equal(s, want_s)
    assert around_q() and around_s()
    for t in DT.values():
        d, around = guarded((R, K), t)
        gq.gq_dequantize_fp8(q, s, rows, out=d)
        assert torch.equal(d, gq.gq_dequantize_fp8(q, s, rows, dtype=t)) and around()


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 7, 7), (9, 256, 8), (17, 33, 16), (100, 1000, 4)])
def test_bytes_around_router_outputs(T, E, k):
    g = torch.Generator("cuda").manual_seed(T)
    x, Wr = torch.randn(T, 72, device="cuda", generator=g), torch.randn(E, 72, device="cuda", generator=g)
    if T > 1:
        x[1, 3] = float("nan")  # a token without experts
    ids, around_ids = guarded((T, k), torch.int32)
    w, around_w = guarded((T, k), torch.float32)
    ws, around_ws = guarded((gq.gq_moe_route_workspace_bytes(T, E),), torch.uint8)
    ws.zero_()
    for _ in range(2):
        gq.gq_moe_route(x, Wr, k, ids=ids, weights=w, workspace=ws)
        want_ids, want_w = gq.gq_moe_route(x, Wr, k)
        assert torch.equal(ids, want_ids) and torch.equal(w, want_w)
        assert around_ids() and around_w() and around_ws()
