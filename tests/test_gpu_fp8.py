"""8-bit blocks and their product against plain 64-bit forms."""
import numpy as np
import pytest
import torch

import bit_gemv_q4_b200 as gq

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def e4m3(v):
    """v (64 bits) rounded to e4m3: three bits after the leading one, steps of 2^-9 below 2^-6."""
    v = np.clip(v, -448.0, 448.0)
    step = 2.0 ** (np.maximum(np.frexp(np.abs(v))[1] - 1, -6) - 3)
    return np.clip(np.rint(v / step) * step, -448.0, 448.0)


def quantized(x, rows):
    """(codes' values, scales) by the rule, quotients in fp32."""
    R, K = x.shape
    rb, kb = -(-R // rows), -(-K // 128)
    p = np.zeros((rb * rows, kb * 128), dtype=np.float32)
    p[:R, :K] = x
    p = p.reshape(rb, rows, kb, 128)
    s = (np.abs(p).max(axis=(1, 3)) / np.float32(448)).astype(np.float32)
    d = s[:, None, :, None]
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.where(d > 0, (p / d).astype(np.float32), np.float32(0)).astype(np.float64)
    return e4m3(q).reshape(rb * rows, kb * 128)[:R, :K], s


def spread(s, rows, R, K):
    return np.repeat(np.repeat(s, rows, axis=0)[:R], 128, axis=1)[:, :K]


@pytest.mark.parametrize("R,K", [(1, 16), (1, 128), (3, 144), (7, 4096), (129, 400), (300, 1040)])
@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("xt", list(DT))
def test_quantize_and_dequantize(R, K, rows, xt):
    g = torch.Generator().manual_seed(R * K)
    x = (torch.randn(R, K, generator=g) * torch.exp(3 * torch.randn(R, 1, generator=g))).to(DT[xt])
    x[0, :16] = 0.0
    if K > 256 and R > 130:
        x[128:, 128:256] = 0.0  # a block of zeros
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    q, s = gq.gq_quantize_fp8(x.cuda(), rows, dev_status=st)
    want, ws = quantized(x.float().numpy(), rows)
    assert int(st.item()) == 0
    assert np.array_equal(s.cpu().numpy(), ws)
    assert np.array_equal(q.float().cpu().numpy().astype(np.float64), want)
    for t in DT.values():  # exact product rounded to fp32, then to the type
        d = gq.gq_dequantize_fp8(q, s, rows, dtype=t)
        v = (want * spread(ws, rows, R, K).astype(np.float64)).astype(np.float32)
        assert torch.equal(d.cpu(), torch.from_numpy(v).to(t))


def test_quantize_extremes():
    x = torch.zeros(4, 256)
    x[0, 5] = 1e-45                       # the scale rounds to zero: codes 0
    x[1, 7] = torch.finfo(torch.float32).max
    x[2] = 448.0
    x[3, 130], x[3, 131] = 3e-38, -1e-40  # a subnormal scale
    q, s = gq.gq_quantize_fp8(x.cuda(), 1)
    want, ws = quantized(x.numpy(), 1)
    assert np.array_equal(s.cpu().numpy(), ws)
    assert np.array_equal(q.float().cpu().numpy().astype(np.float64), want)
    assert float(s[0, 0]) == 0.0 and not q[0].float().any()


def test_quantize_codes_at_the_middles():
    # quotients at, and one to five fp32 steps beside, every middle between two codes; zeros and the
    # evenly spaced small codes too
    mids = [(1 + (2 * m + 1) / 16) * 2.0 ** e for e in range(-6, 9) for m in range(8)]
    mids += [(2 * m + 1) * 2.0 ** -10 for m in range(8)]
    v = np.array([m for m in mids if m < 448], dtype=np.float32)
    near = np.concatenate([(v.view(np.int32) + d).view(np.float32) for d in range(-5, 6)])
    for s in (1.0, 3.0, 0.1, 7e-3, 1.7e-36, 3e34):
        row = (near.astype(np.float64) * s).astype(np.float32)
        n = -(-(row.size + 1) // 127)
        x = np.zeros((n, 128), dtype=np.float32)
        x[:, 0] = np.float32(448 * s)                # sets the scale near s
        x[:, 1:].reshape(-1)[:] = 0
        x[:, 1:] = np.resize(row, n * 127).reshape(n, 127)
        q, sc = gq.gq_quantize_fp8(torch.from_numpy(x).cuda(), 1)
        want, ws = quantized(x, 1)
        assert np.array_equal(sc.cpu().numpy(), ws)
        assert np.array_equal(q.float().cpu().numpy().astype(np.float64), want)


@pytest.mark.parametrize("rows", [1, 128])
def test_quantize_reports_nonfinite_and_keeps_other_blocks(rows):
    x = torch.randn(130, 272, device="cuda")
    q0, s0 = gq.gq_quantize_fp8(x, rows)
    for bad in (float("nan"), float("inf")):
        y = x.clone()
        y[129, 200] = bad
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        q, s = gq.gq_quantize_fp8(y, rows, dev_status=st)
        assert int(st.item()) == gq.GQ_DEV_NONFINITE
        keep = torch.ones(130, 272, dtype=torch.bool, device="cuda")
        keep[129 if rows == 1 else slice(128, 130), 128:256] = False
        assert torch.equal(q.view(torch.uint8)[keep], q0.view(torch.uint8)[keep])


def operands(M, K, B, seed):
    g = torch.Generator().manual_seed(seed)
    W = torch.randn(M, K, generator=g) * 0.02 * torch.exp(torch.randn(M, 1, generator=g) / 2)
    X = torch.randn(B, K, generator=g) * torch.exp(torch.randn(B, 1, generator=g))
    return gq.gq_quantize_fp8(W.cuda(), 128) + gq.gq_quantize_fp8(X.cuda(), 1)


def check(Y, W, ws, X, xs):
    """Exact products; 128 of them and the accumulator in at most 140 additions, each cut to 24 bits
    (a whole step, 2^-23); then one fused multiply-add for each group, two roundings in its factor
    and, for cut tiles, a few more additions: (groups + 8) half steps."""
    (M, K), B = W.shape, X.shape[0]
    Wd = W.double() * torch.from_numpy(spread(ws.cpu().numpy(), 128, M, K)).cuda().double()
    Xd = X.double() * torch.from_numpy(spread(xs.cpu().numpy(), 1, B, K)).cuda().double()
    want, mag = Xd @ Wd.T, Xd.abs() @ Wd.abs().T
    groups = -(-K // 128)
    allow = (140 * 2.0 ** -23 + (groups + 8) * 2.0 ** -24) * mag
    allow += torch.finfo(Y.dtype).eps / 2 * (want.abs() + allow) + 2.0 ** -25
    err = (Y.double() - want).abs()
    assert bool((err <= allow).all()), float((err / allow).max())


@pytest.mark.parametrize("M,K,B,yt", [
    (1, 16, 1, "f32"), (128, 128, 128, "f32"), (5, 48, 3, "bf16"), (300, 144, 130, "f32"),
    (200, 4096, 100, "f32"), (1000, 2064, 67, "f16"), (129, 4096, 128, "bf16"), (2000, 512, 65, "f32"),
    (70, 11008, 7, "f32"), (33, 1040, 16, "f32"), (64, 2048, 17, "f32"), (6200, 4096, 16, "bf16"),
    (700, 2048, 600, "f32"), (12000, 256, 300, "bf16"), (2571, 272, 1025, "f32"), (2572, 272, 1025, "f32"),
    (4096, 4096, 1, "bf16"), (1000, 2064, 9, "f16"), (129, 4096, 33, "f32"), (2000, 512, 64, "f32"),
    (11000, 256, 37, "f16"), (257, 8192, 65, "bf16"), (4096, 1024, 500, "bf16"),
    (520, 400, 4000, "f32"), (6001, 384, 1300, "f16"), (9000, 128, 2500, "f32"), (4095, 640, 2049, "bf16"),
])
def test_gemm(M, K, B, yt):
    W, ws, X, xs = operands(M, K, B, M + K + B)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    Y = gq.gq_gemm_fp8(W, ws, X, xs, y_dtype=DT[yt], dev_status=st)
    check(Y, W, ws, X, xs)
    assert int(st.item()) == 0
    assert torch.equal(gq.gq_gemm_fp8(W, ws, X, xs, y_dtype=DT[yt]), Y)  # the same bits again


def test_gemm_guards_and_one_workspace_for_all_sizes():
    cases = [(1000, 2064, 9), (129, 4096, 33), (300, 144, 130), (200, 4096, 100), (4096, 256, 1)]
    need = max(gq.gq_gemm_fp8_workspace_bytes(*c) for c in cases)
    buf = torch.zeros(need + 512, dtype=torch.uint8, device="cuda")
    buf[need:] = 0xA5
    for M, K, B in cases * 2:
        W, ws, X, xs = operands(M, K, B, M)
        out = torch.full((B + 16, M), 7.0, device="cuda")
        y = out.view(-1)[8 * M:8 * M + B * M]
        gq.gq_gemm_fp8(W, ws, X, xs, out=y, workspace=buf[:need])
        check(y.view(B, M), W, ws, X, xs)
        assert bool((out[:8] == 7).all()) and bool((out[B + 8:] == 7).all())
    assert bool((buf[need:] == 0xA5).all())


def test_gemm_nan_code_stays_in_its_token_and_row():
    W, ws, X, xs = operands(400, 512, 70, 3)
    good = gq.gq_gemm_fp8(W, ws, X, xs, y_dtype=torch.float32)
    X.view(torch.uint8)[41, 300] = 0x7F
    y = gq.gq_gemm_fp8(W, ws, X, xs, y_dtype=torch.float32)
    assert not torch.isfinite(y[41]).any()
    keep = torch.arange(70, device="cuda") != 41
    assert torch.equal(y[keep], good[keep])


def test_quantize_then_gemm_captured_and_on_another_stream():
    M, K, B = 1030, 1040, 50
    g = torch.Generator().manual_seed(1)
    W, ws = gq.gq_quantize_fp8((torch.randn(M, K, generator=g) * 0.02).cuda(), 128)
    x = torch.randn(B, K, generator=g).bfloat16().cuda()

    def step():
        q, s = gq.gq_quantize_fp8(x, 1)
        return gq.gq_gemm_fp8(W, ws, q, s, flags=gq.GQ_GEMV_PDL, y_dtype=torch.float32), q, s

    y, q, s = step()
    check(y, W, ws, q, s)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        y2 = step()[0]
    st.synchronize()
    assert torch.equal(y, y2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y3 = step()[0]
    for seed in (2, 3):
        x.copy_(torch.randn(B, K, generator=torch.Generator().manual_seed(seed)).bfloat16())
        graph.replay()
        y4, q, s = step()
        torch.cuda.synchronize()
        assert torch.equal(y3, y4)
        check(y3, W, ws, q, s)


def test_gemm_agrees_with_the_dequantized_product():
    W, ws, X, xs = operands(384, 640, 20, 5)
    Wd, Xd = gq.gq_dequantize_fp8(W, ws, 128), gq.gq_dequantize_fp8(X, xs, 1)
    y = gq.gq_gemm_fp8(W, ws, X, xs, y_dtype=torch.float32)
    want = Xd.double() @ Wd.double().T
    # the decoded values carry one more rounding each
    assert bool(((y.double() - want).abs() <= 160 * 2.0 ** -23 * (Xd.double().abs() @ Wd.double().abs().T)).all())
