"""8-bit blocks on the CPU: sizes, and refusals before any launch."""
import pytest
import torch

import bit_gemv_q4_b200 as gq

INVALID, SHAPE, ALIGN, DTYPE, WORKSPACE = 1, 2, 3, 4, 9
A = 0x10000000  # aligned fake device address


def test_sizes():
    assert gq.gq_fp8_scales(1, 16, 1) == 1 and gq.gq_fp8_scales(7, 4096, 1) == 7 * 32
    assert gq.gq_fp8_scales(129, 144, 128) == 4 and gq.gq_fp8_scales(0, 128, 1) == 0
    for bad in ((4, 24, 1), (4, 128, 2), (-1, 128, 1), (4, 1 << 25, 1), (1 << 31, 16, 1)):
        assert gq.gq_fp8_scales(*bad) == 0
    assert gq.gq_gemm_fp8_workspace_bytes(0, 128, 1) == 0
    assert gq.gq_gemm_fp8_workspace_bytes(128, 24, 1) == 0
    assert gq.gq_gemm_fp8_workspace_bytes(4096, 4096, 1) == 0      # few tokens need none
    assert gq.gq_gemm_fp8_workspace_bytes(4096, 4096, 100) > 0


def test_quantize_refusals():
    def q(x=A, xt=0, R=4, K=128, rows=1, out=A, s=A, st=None):
        return gq.lib.gq_quantize_fp8(x, xt, R, K, rows, out, s, st, None)

    assert q(xt=3) == DTYPE
    assert q(R=-1) == INVALID and q(K=-16) == INVALID and q(rows=2) == INVALID and q(rows=0) == INVALID
    assert q(K=24) == SHAPE and q(K=1 << 25) == SHAPE and q(R=1 << 31) == SHAPE
    assert q(x=None) == INVALID and q(out=None) == INVALID and q(s=None) == INVALID
    assert q(x=A + 8) == ALIGN and q(out=A + 4) == ALIGN and q(s=A + 4) == ALIGN and q(st=A + 2) == ALIGN
    assert q(R=0) == 0 and q(K=0) == 0

    def d(qq=A, s=A, R=4, K=128, rows=128, out=A, t=0):
        return gq.lib.gq_dequantize_fp8(qq, s, R, K, rows, out, t, None)

    assert d(t=5) == DTYPE and d(rows=64) == INVALID and d(K=8) == SHAPE
    assert d(qq=None) == INVALID and d(s=None) == INVALID and d(out=None) == INVALID
    assert d(qq=A + 2) == ALIGN and d(out=A + 8) == ALIGN
    assert d(R=0) == 0


def test_gemm_refusals():
    ok = dict(W=A, ws=A, M=256, K=128, X=A, xs=A, B=4, Y=A, yt=0, work=A, wb=1 << 26, flags=0, st=None)

    def call(**kw):
        a = dict(ok, **kw)
        return gq.lib.gq_gemm_fp8(a["W"], a["ws"], a["M"], a["K"], a["X"], a["xs"], a["B"], a["Y"], a["yt"],
                                  a["work"], a["wb"], a["flags"], a["st"], None)

    for n in ("M", "K", "B"):
        assert call(**{n: -1}) == INVALID
    assert call(yt=3) == DTYPE and call(flags=2) == INVALID
    assert call(K=120) == SHAPE and call(K=1 << 25) == SHAPE and call(B=1 << 31) == SHAPE
    for n in ("W", "ws", "X", "xs", "Y"):
        assert call(**{n: None}) == INVALID
        assert call(**{n: A + 4}) == ALIGN
    assert call(st=A + 1) == ALIGN
    need = gq.gq_gemm_fp8_workspace_bytes(256, 4096, 100)
    ok["K"] = 4096
    assert call(B=100, work=None) == WORKSPACE and call(B=100, wb=need - 1) == WORKSPACE
    assert call(B=100, work=A + 16) == ALIGN
    assert call(M=0) == 0 and call(B=0) == 0


def test_binding_refusals():
    x = torch.zeros(4, 128)
    with pytest.raises(ValueError):
        gq.gq_quantize_fp8(x, 64)
    with pytest.raises(TypeError):
        gq.gq_quantize_fp8(x.double(), 1)
    q, s = torch.zeros(4, 128).to(torch.float8_e4m3fn), torch.zeros(4, 1)
    with pytest.raises(TypeError):
        gq.gq_dequantize_fp8(q.view(torch.uint8), s, 1)
    with pytest.raises(ValueError):  # too few scales
        gq.gq_dequantize_fp8(q, s[:3], 1)
    with pytest.raises(ValueError):  # another K
        gq.gq_gemm_fp8(q, s, torch.zeros(2, 256).to(torch.float8_e4m3fn), torch.zeros(2, 2))
