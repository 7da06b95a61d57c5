"""Bounded waits that run out inside the newer kernels (something that never
comes, about 1 ms): they report GQ_DEV_TIMEOUT, the context stays usable, and the
calls after them on the same workspace give the bits they gave before."""
import pytest
import torch

import bit_gemv_q4_b200 as gq
from gpu_helpers import Q40
from test_gpu_fp8 import check, operands
from test_gpu_moe import Layer, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("workspace", ["auto", "own"])
@pytest.mark.parametrize("T", [1, 4, 33])
def test_layer_after_a_barrier_that_was_not_passed(T, workspace):
    m = Layer(Q40, 8, 512, 192)
    x, ids, w = inputs(T, 512, 8, 3, "f16", seed=T)
    ws = workspace
    if ws == "own":
        ws = torch.zeros(gq.gq_moe_workspace_bytes(gq.GQ_FMT_Q4_0, 512, 192, 33, 3), dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = m(x, ids, w, y_dtype=torch.float32, workspace=ws)
    big, y = x * 1000, torch.empty_like(x)  # h a million times as large
    for n in range(3):
        for _ in range(n + 1):
            st.zero_()
            gq.gq_selftest_moe_timeout(m.gate, m.up, m.down, 8, 192, big, ids, w, y, st, workspace=ws)
            torch.cuda.synchronize()
            assert int(st.item()) == gq.GQ_DEV_TIMEOUT
            assert gq.gq_status_from_dev(int(st.item())) == 7
        st.zero_()
        got = m(x, ids, w, y_dtype=torch.float32, workspace=ws, dev_status=st)
        assert int(st.item()) == 0
        assert torch.equal(got, want)
    m.check(got, x, ids, w)


def test_layer_selftest_needs_a_status_word():
    m = Layer(Q40, 8, 512, 192)
    x, ids, w = inputs(2, 512, 8, 3, "f16", seed=1)
    with pytest.raises(gq.GQError):
        gq.gq_selftest_moe_timeout(m.gate, m.up, m.down, 8, 192, x, ids, w, torch.empty_like(x), None)


@pytest.mark.parametrize("M,K,B", [
    (129, 4096, 128),                     # tiles cut along K, and the launch that adds the pieces
    (300, 144, 130), (2000, 16, 40),      # whole tiles, of two groups and of one
    (2571, 272, 1025), (9000, 400, 2500),  # pairs of CTAs
])
def test_product_after_a_stage_that_was_never_filled(M, K, B):
    W, ws, X, xs = operands(M, K, B, M + K)
    want = gq.gq_gemm_fp8(W, ws, X, xs, y_dtype=torch.float32)
    check(want, W, ws, X, xs)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    rows = torch.full((B + 2, M), 7.0, device="cuda")
    around = rows.view(-1)[: 8 * ((M + 7) // 8)], rows.view(-1)[8 * ((M + 7) // 8) + B * M:]
    Y = rows.view(-1)[8 * ((M + 7) // 8):][:B * M].view(B, M)
    for _ in range(3):
        st.zero_()
        gq.gq_selftest_gemm_fp8_timeout(W, ws, X, xs, Y, st)
        torch.cuda.synchronize()
        assert int(st.item()) == gq.GQ_DEV_TIMEOUT
        assert all(bool((a == 7).all()) for a in around)
        st.zero_()
        got = gq.gq_gemm_fp8(W, ws, X, xs, y_dtype=torch.float32, dev_status=st)
        assert int(st.item()) == 0 and torch.equal(got, want)


def test_product_selftest_refuses_few_tokens():
    W, ws, X, xs = operands(256, 128, 4, 1)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    with pytest.raises(gq.GQError):
        gq.gq_selftest_gemm_fp8_timeout(W, ws, X, xs, torch.empty(4, 256, device="cuda"), st)
