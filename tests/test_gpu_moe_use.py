"""The router, the expert layer and the 8-bit operators as a program uses them:
together, on several streams at once, captured, by keyword, and at the largest
sizes.  Values are held against tests/moe_ref.py or against the same call done
alone, whose bits have to be the same."""
import numpy as np
import pytest
import torch

import bit_gemv_q4_b200 as gq
from gpu_helpers import KSB, Q40
from test_gpu_fp8 import check as check_gemm
from test_gpu_moe import Layer, inputs

pytestmark = pytest.mark.gpu


def test_a_block_of_all_of_them_captured_and_eager():
    m = Layer(Q40, 16, 256, 704)
    g = torch.Generator().manual_seed(2)
    Wr = torch.randn(16, 256, generator=g).bfloat16().cuda()
    Wh, hs = gq.gq_quantize_fp8((torch.randn(520, 256, generator=g) * 0.05).cuda(), 128)
    x = torch.randn(33, 256, generator=g).bfloat16().cuda()

    def block():
        ids, w = gq.gq_moe_route(x, Wr, 4, flags=gq.GQ_ROUTE_NORM)
        y = m(x, ids, w, y_dtype=torch.bfloat16, flags=gq.GQ_GEMV_PDL)
        q, s = gq.gq_quantize_fp8(y, 1)
        return ids, w, y, q, s, gq.gq_gemm_fp8(Wh, hs, q, s, y_dtype=torch.float32, flags=gq.GQ_GEMV_PDL)

    block()  # one call outside the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = block()
    for seed in (5, 6, 7):
        x.copy_(torch.randn(33, 256, generator=torch.Generator().manual_seed(seed)).bfloat16())
        graph.replay()
        eager = block()
        torch.cuda.synchronize()
        for a, b in zip(kept, eager):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        ids, w, y, q, s, z = kept
        m.check(y, x, ids, w)
        check_gemm(z, Wh, hs, q, s)


def test_two_streams_at_once():
    a, b = Layer(Q40, 16, 256, 704), Layer(KSB, 4, 2304, 512)
    xa, ia, wa = inputs(9, 256, 16, 4, "f16", seed=1)
    xb, ib, wb = inputs(1, 2304, 4, 3, "bf16", seed=2)
    W, ws = gq.gq_quantize_fp8(torch.randn(300, 2048, device="cuda"), 128)
    X, xs = gq.gq_quantize_fp8(torch.randn(40, 2048, device="cuda"), 1)
    Wr = torch.randn(64, 256, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")

    def one():
        return (*gq.gq_moe_route(xa, Wr, 5), a(xa, ia, wa, dev_status=st),
                gq.gq_gemm_fp8(W, ws, X, xs, dev_status=st))

    def two():
        return (gq.gq_gemm_fp8(W, ws, X, xs, dev_status=st), b(xb, ib, wb, dev_status=st),
                *gq.gq_moe_route(xa, Wr, 5), a(xa, ia, wa, dev_status=st))

    want = one(), two()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        with torch.cuda.stream(s1):
            one_now = one()
        with torch.cuda.stream(s2):
            two_now = two()
        got.append((one_now, two_now))
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    for pair in got:
        for outs, ref in zip(pair, want):
            for o, r in zip(outs, ref):
                assert torch.equal(o, r)


def test_two_graphs_replayed_at_once():
    m = Layer(Q40, 8, 512, 192)
    W, ws = gq.gq_quantize_fp8(torch.randn(300, 2048, device="cuda"), 128)
    X, xs = gq.gq_quantize_fp8(torch.randn(40, 2048, device="cuda"), 1)
    Wr = torch.randn(8, 512, device="cuda")
    graphs = []
    for T in (1, 5):
        x = torch.randn(T, 512, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            ids, w = gq.gq_moe_route(x, Wr, 3)
            out = ids, w, m(x, ids, w, flags=gq.GQ_GEMV_PDL), gq.gq_gemm_fp8(W, ws, X, xs)
        graphs.append((graph, x, out, torch.cuda.Stream()))
    for n in range(10):
        for graph, x, out, s in graphs:
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for graph, x, out, s in graphs:
            ids, w = gq.gq_moe_route(x, Wr, 3)
            for o, r in zip(out, (ids, w, m(x, ids, w), gq.gq_gemm_fp8(W, ws, X, xs))):
                assert torch.equal(o, r)
            x.mul_(-1.25)


def test_a_named_stream_eager_and_under_capture():
    m = Layer(Q40, 8, 512, 192)
    x, ids, w = inputs(5, 512, 8, 3, "f16", seed=4)
    want = m(x, ids, w)
    s = torch.cuda.Stream()
    out = torch.empty_like(want)
    torch.cuda.synchronize()
    m(x, ids, w, out=out, stream=s)          # a torch stream, and a raw handle
    s.synchronize()
    assert torch.equal(out, want)
    out.zero_()
    torch.cuda.synchronize()
    m(x, ids, w, out=out, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(out, want)
    # a stream that joined a capture, named while another one is current: the captured call gets a
    # workspace of its own, not the one that eager calls on that stream keep using
    graph = torch.cuda.CUDAGraph()
    out.zero_()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        s.wait_stream(torch.cuda.current_stream())
        m(x, ids, w, out=out, stream=s)
        torch.cuda.current_stream().wait_stream(s)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    out.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        eager = [m(x, ids, w) for _ in range(10)]
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and all(torch.equal(e, want) for e in eager)


def test_calls_by_keyword():
    m = Layer(Q40, 8, 512, 192)
    x, ids, w = inputs(5, 512, 8, 3, "f16", seed=4)
    Wr = torch.randn(8, 512, device="cuda")
    for a, b in zip(gq.gq_moe_route(x=x, Wr=Wr, k=2), gq.gq_moe_route(x, Wr, 2)):
        assert torch.equal(a, b)
    y = gq.gq_moe_q4_0_tiled(gate=m.gate, up=m.up, down=m.down, E=8, I=192, x=x, ids=ids, weights=w)
    assert torch.equal(y, m(x, ids, w))
    q, s = gq.gq_quantize_fp8(x=x, rows=1)
    assert torch.equal(gq.gq_dequantize_fp8(q=q, scales=s, rows=1), gq.gq_dequantize_fp8(q, s, 1))


def test_strided_inputs_are_refused():
    m = Layer(Q40, 8, 512, 192)
    x, ids, w = inputs(5, 512, 8, 3, "f16", seed=4)
    wide = torch.zeros(5, 1024, dtype=torch.float16, device="cuda")
    for bad in ((wide[:, :512], ids, w), (x, ids.T.contiguous().T, w), (x, ids, w.T.contiguous().T)):
        with pytest.raises(ValueError):
            m(*bad)
    with pytest.raises(ValueError):
        gq.gq_moe_route(wide[:, :512], torch.zeros(8, 512, device="cuda"), 2)
    with pytest.raises(ValueError):
        gq.gq_quantize_fp8(wide[:, :512], 1)
    with pytest.raises(gq.GQError):  # rows that begin at 2 bytes past a 16-byte boundary
        gq.gq_quantize_fp8(wide.view(-1)[1:1 + 512].view(1, 512), 1)
    q, s = gq.gq_quantize_fp8(x, 1)
    W, ws = gq.gq_quantize_fp8(torch.zeros(64, 1024, device="cuda"), 128)
    with pytest.raises(ValueError):
        gq.gq_gemm_fp8(W[:, :512], ws[:, :4].contiguous(), q, s)


def test_empty_calls():
    m = Layer(Q40, 8, 512, 192)
    x = torch.empty(0, 512, dtype=torch.float16, device="cuda")
    ids, w = gq.gq_moe_route(x, torch.zeros(8, 512, device="cuda"), 3)
    assert ids.shape == (0, 3) and w.shape == (0, 3)
    assert m(x, ids, w).shape == (0, 512)
    none = torch.empty(4, 0, device="cuda")  # no slots: zeros
    x = torch.ones(4, 512, dtype=torch.float16, device="cuda")
    assert not m(x, none.int(), none).any()
    q, s = gq.gq_quantize_fp8(x[:0], 1)
    W, ws = gq.gq_quantize_fp8(torch.zeros(64, 512, device="cuda"), 128)
    assert gq.gq_gemm_fp8(W, ws, q, s).shape == (0, 64)


def test_route_bias_of_infinities_and_nan():
    x = torch.randn(9, 64, device="cuda")
    Wr = torch.randn(40, 64, device="cuda")
    bias = torch.zeros(40, device="cuda")
    bias[3], bias[17] = float("-inf"), float("inf")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ids, w = gq.gq_moe_route(x, Wr, 16, bias=bias, flags=gq.GQ_ROUTE_SIGMOID, dev_status=st)
    assert int(st.item()) == 0
    assert bool((ids[:, 0] == 17).all()) and not bool((ids == 3).any())
    z = torch.sigmoid(x.double() @ Wr.double().T)
    # a sigmoid's value rounded to 32 bits, and the product with scale 1
    assert bool(((w.double() - z.gather(1, ids.long())).abs() <= 2.0 ** -23 * w).all())
    bias[20] = float("nan")
    ids, w = gq.gq_moe_route(x, Wr, 16, bias=bias, flags=gq.GQ_ROUTE_SIGMOID, dev_status=st)
    assert int(st.item()) == gq.GQ_DEV_NONFINITE
    assert bool((ids == -1).all()) and not w.any()


def test_route_most_tokens_and_a_long_row():
    x = torch.zeros(65536, 8, device="cuda")
    x[:, 0] = torch.arange(65536, device="cuda") % 7 - 3.0
    Wr = torch.zeros(6, 8, device="cuda")
    Wr[:, 0] = torch.tensor([0.5, -1.0, 2.0, -3.0, 1.0, 0.0])
    ids, _ = gq.gq_moe_route(x, Wr, 2)
    z = x[:, :1].double() * Wr[:, 0].double()
    want = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :2]
    assert torch.equal(ids.long(), want)
    H = 1 << 20
    x, Wr = torch.randn(2, H, device="cuda"), torch.randn(40, H, device="cuda") / 1024
    ids, _ = gq.gq_moe_route(x, Wr, 16)
    z = x.double() @ Wr.double().T
    assert torch.equal(ids.long(), torch.sort(z, dim=1, descending=True, stable=True).indices[:, :16])


def test_layer_most_experts_tokens_and_slots():
    m = Layer(Q40, 1024, 64, 64)
    x, ids, w = inputs(64, 64, 1024, 16, "bf16", seed=11)
    m.check(m(x, ids, w, y_dtype=torch.float32), x, ids, w)
    ids[:] = 1023  # every pair the same expert
    m.check(m(x, ids, w, y_dtype=torch.float32), x, ids, w)


@pytest.mark.parametrize("fmt,E,H,I", [(Q40, 110, 4096, 11008), (KSB, 512, 4096, 2048)])
def test_layer_expert_past_two_to_the_31_bytes(fmt, E, H, I):
    # one expert's storage copied to every place; the last one's place begins past 2^31 bytes
    code = gq.GQ_FMT_Q4_0 if fmt == Q40 else gq.GQ_FMT_KSB
    one = []
    for seed, (R, K) in enumerate(((I, H), (I, H), (H, I))):
        g = torch.Generator(device="cuda").manual_seed(seed)
        v = torch.randn(R, K, device="cuda", generator=g) * 0.02
        quantize = gq.gq_quantize_q4_0 if fmt == Q40 else gq.gq_quantize_ksb
        one.append(gq.gq_repack(code, quantize(v.view(-1)), R, K))
    stacks = [torch.zeros(E, t.numel(), dtype=torch.uint8, device="cuda") for t in one]
    for t, s in zip(one, stacks):
        s[E - 1] = t
    assert (E - 1) * one[0].numel() > 1 << 31
    call = gq.gq_moe_q4_0_tiled if fmt == Q40 else gq.gq_moe_ksb_tiled
    for T in (1, 3):
        x = torch.randn(T, H, device="cuda", dtype=torch.bfloat16)
        w = torch.rand(T, 2, device="cuda")
        ids = torch.tensor([[E - 1, -1]] * T, dtype=torch.int32, device="cuda")
        first = torch.tensor([[0, -1]] * T, dtype=torch.int32, device="cuda")
        big = call(*(s.view(-1) for s in stacks), E, I, x, ids, w)
        small = call(*one, 1, I, x, first, w)
        assert bool(big.any()) and torch.equal(big, small)


def test_eight_bits_past_two_to_the_31():
    R, K = 200_001, 11008  # 2.2e9 values
    x = torch.zeros(R, K, dtype=torch.bfloat16, device="cuda")
    tail = torch.randn(200, K, device="cuda").bfloat16()
    x[-200:] = tail
    for rows in (1, 128):
        q, s = gq.gq_quantize_fp8(x, rows)
        keep = 200 if rows == 1 else 200 - (128 - (R - 200) % 128)  # rows of whole blocks of the tail
        tq, ts = gq.gq_quantize_fp8(tail[200 - keep:], rows)
        assert torch.equal(q[-keep:].view(torch.uint8), tq.view(torch.uint8))
        assert torch.equal(s[-ts.shape[0]:], ts) and not q[:1000].float().any()
    d = gq.gq_dequantize_fp8(q, s, 128, dtype=torch.bfloat16)
    assert torch.equal(d[-keep:], gq.gq_dequantize_fp8(tq, ts, 128, dtype=torch.bfloat16))
    del d, x
    for B in (3, 40, 300):  # a weight matrix of 2.2 GB
        X, xs = gq.gq_quantize_fp8(torch.randn(B, K, device="cuda"), 1)
        Y = gq.gq_gemm_fp8(q, s, X, xs, y_dtype=torch.float32)
        check_gemm(Y[:, -keep:].contiguous(), tq, ts, X, xs)
        assert not Y[:, :1000].any()
    del q, Y
    W, ws = gq.gq_quantize_fp8(torch.randn(20_000, 128, device="cuda"), 128)
    X, xs = gq.gq_quantize_fp8(torch.randn(110_000, 128, device="cuda"), 1)
    Y = gq.gq_gemm_fp8(W, ws, X, xs)  # 2.2e9 outputs
    check_gemm(Y[-200:], W, ws, X[-200:], xs[-200:])


def test_gemm_with_no_columns_is_zeros():
    W = torch.empty(64, 0, dtype=torch.float8_e4m3fn, device="cuda")
    X = torch.empty(3, 0, dtype=torch.float8_e4m3fn, device="cuda")
    none = torch.empty(0, device="cuda")
    out = torch.full((3, 64), 7.0, device="cuda")
    gq.gq_gemm_fp8(W, none, X, none, out=out)
    assert not out.any()


def test_layer_writes_over_its_input():
    # y may be x itself: every x is read before the first y is written
    m = Layer(Q40, 8, 512, 192)
    for T in (1, 7):
        x, ids, w = inputs(T, 512, 8, 3, "f16", seed=T)
        want = m(x, ids, w)
        m(x, ids, w, out=x)
        assert torch.equal(x, want)
        assert np.isfinite(x.float().cpu().numpy()).all()


def test_buffers_that_the_next_call_writes_again():
    # calls may start early: each has to wait for the one before it before it writes what that one reads
    m = Layer(Q40, 8, 512, 192)
    Wr = torch.randn(8, 512, device="cuda")
    W, ws = gq.gq_quantize_fp8(torch.randn(1030, 512, device="cuda"), 128)
    xs = [torch.randn(T, 512, device="cuda", dtype=torch.bfloat16) for T in (40, 3, 40, 17, 1, 40) for _ in range(4)]
    ids, w = torch.empty(40 * 3, dtype=torch.int32, device="cuda"), torch.empty(40 * 3, device="cuda")
    q = torch.empty(40, 512, dtype=torch.float8_e4m3fn, device="cuda")
    s, y = torch.empty(40, 4, device="cuda"), torch.empty(40, 512, dtype=torch.bfloat16, device="cuda")

    def chain(x, sync):
        T = x.shape[0]
        step = torch.cuda.synchronize if sync else lambda: None
        i, v = gq.gq_moe_route(x, Wr, 3, ids=ids[:T * 3].view(T, 3), weights=w[:T * 3].view(T, 3))
        step()
        m(x, i, v, out=y[:T])
        step()
        gq.gq_quantize_fp8(y[:T], 1, out=q[:T], scales=s[:T])
        step()
        out = gq.gq_gemm_fp8(W, ws, q[:T], s[:T])
        step()
        return out

    want = [chain(x, True) for x in xs]
    for _ in range(5):
        got = [chain(x, False) for x in xs]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
