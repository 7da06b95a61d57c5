"""The router and the 4-bit expert layer against plain 64-bit forms; the
allowed errors are those of tests/moe_ref.py, derived from the arithmetic."""
import numpy as np
import pytest
import torch

import bit_gemv_q4_b200 as gq
import oracle
from gpu_helpers import KSB, Q40
import moe_ref

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_cache = {}


def stack(fmt, E, R, K, seed):
    key = (fmt, E, R, K, seed)
    if key not in _cache:
        q, dec, d = moe_ref.experts(fmt, E, R, K, seed)
        code = gq.GQ_FMT_Q4_0 if fmt == Q40 else gq.GQ_FMT_KSB
        _cache[key] = gq.gq_repack(code, torch.from_numpy(q).cuda(), E * R, K), (dec, d)
    return _cache[key]


class Layer:
    def __init__(self, fmt, E, H, I):
        self.fmt, self.E, self.H, self.I = fmt, E, H, I
        self.gate, self.g = stack(fmt, E, I, H, 1)
        self.up, self.u = stack(fmt, E, I, H, 2)
        self.down, self.d = stack(fmt, E, H, I, 3)
        self.call = gq.gq_moe_q4_0_tiled if fmt == Q40 else gq.gq_moe_ksb_tiled

    def __call__(self, x, ids, w, **kw):
        return self.call(self.gate, self.up, self.down, self.E, self.I, x, ids, w, **kw)

    def check(self, y, x, ids, w):
        want, allow = moe_ref.layer(self.g, self.u, self.d, x.double().cpu().numpy(), ids.cpu().numpy(),
                                    w.double().cpu().numpy(), x.dtype == torch.float32,
                                    torch.finfo(y.dtype).eps / 2)
        err = np.abs(y.double().cpu().numpy() - want)
        assert np.all(np.isfinite(err)) and np.all(err <= allow), float((err / allow).max())


def inputs(T, H, E, k, xt, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(T, H, generator=g) * spread).to(DT[xt])
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32)
    w = torch.rand(T, k, generator=g) + 0.1
    return x.cuda(), ids.cuda(), w.cuda()


@pytest.mark.parametrize("fmt,E,H,I,T,k,xt,yt", [
    (Q40, 4, 64, 64, 1, 1, "f16", "f16"),            # one unit per row group
    (Q40, 4, 64, 64, 1, 1, "f32", "f32"),
    (KSB, 3, 256, 256, 1, 2, "f16", "f32"),
    (Q40, 8, 512, 192, 1, 2, "bf16", "bf16"),
    (Q40, 8, 2112, 320, 3, 2, "f16", "f32"),          # a short last tile in both products
    (KSB, 4, 2304, 512, 2, 3, "bf16", "f16"),
    (Q40, 16, 256, 704, 16, 4, "f32", "f32"),         # two column tiles, two columns a token
    (Q40, 2, 256, 2176, 20, 2, "f16", "f16"),         # more tokens than a segment takes
    (KSB, 2, 512, 256, 64, 2, "bf16", "f32"),
    (Q40, 64, 128, 128, 64, 16, "f16", "bf16"),       # most tokens and slots
    (Q40, 200, 128, 64, 7, 5, "bf16", "f32"),         # experts beyond one lane each
    (Q40, 2, 16384, 64, 2, 1, "f32", "f32"),          # widest rows
    (Q40, 2, 64, 16384, 5, 2, "f16", "f32"),
])
def test_layer_shapes(fmt, E, H, I, T, k, xt, yt):
    m = Layer(fmt, E, H, I)
    x, ids, w = inputs(T, H, E, k, xt, seed=T + H)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = m(x, ids, w, y_dtype=DT[yt], dev_status=st)
    m.check(y, x, ids, w)
    assert int(st.item()) == 0
    assert torch.equal(m(x, ids, w, y_dtype=DT[yt]), y)  # the same bits again


@pytest.mark.parametrize("fmt,E,H,I,k,xt,yt", [
    (Q40, 16, 512, 704, 6, "bf16", "bf16"), (Q40, 20, 256, 192, 16, "f16", "f32"),
    (KSB, 16, 256, 512, 8, "f32", "f32"), (Q40, 4, 64, 64, 3, "f16", "f16"),
    (Q40, 2, 64, 16384, 2, "f16", "f32"),       # a slot's h is too wide for the others to stay beside it
    (Q40, 3, 2112, 320, 2, "bf16", "f32"),
])
def test_layer_single_token(fmt, E, H, I, k, xt, yt):
    m = Layer(fmt, E, H, I)
    x, ids, w = inputs(1, H, E, k, xt, seed=I + k)
    w[0, 0] = -3.0                               # weights of any sign and size
    if k > 2:
        w[0, 1] = 1e-4
    for change in (None, "skip", "twice", "none"):
        if change == "skip":
            ids[0, k // 2] = -1
        if change == "twice":
            ids[0, -1] = ids[0, 0]
        if change == "none":
            ids[:] = -1
        y = m(x, ids, w, y_dtype=DT[yt])
        m.check(y, x, ids, w)
        assert torch.equal(m(x, ids, w, y_dtype=DT[yt]), y)
    assert not y.any()


def test_layer_single_tokens_and_batches_in_turn_on_one_workspace():
    m = Layer(Q40, 8, 512, 192)
    ws = torch.zeros(gq.gq_moe_workspace_bytes(gq.GQ_FMT_Q4_0, 512, 192, 9, 3), dtype=torch.uint8, device="cuda")
    for n, T in enumerate((1, 1, 4, 1, 9, 9, 1, 1, 1, 2)):
        x, ids, w = inputs(T, 512, 8, 3, "f16", seed=n, spread=10.0 ** (n % 5 - 2))
        m.check(m(x, ids, w, y_dtype=torch.float32, workspace=ws), x, ids, w)


@pytest.mark.parametrize("spread", [1e-6, 1e4])
def test_layer_scales_of_activations(spread):
    m = Layer(Q40, 8, 512, 192)
    for xt in ("bf16", "f32"):
        x, ids, w = inputs(4, 512, 8, 2, xt, seed=9, spread=spread)
        x[1] *= 1e-3
        m.check(m(x, ids, w, y_dtype=torch.float32), x, ids, w)


def test_layer_ids_that_name_nothing():
    m = Layer(Q40, 8, 512, 192)
    x, ids, w = inputs(5, 512, 8, 3, "f16", seed=4)
    ids[0] = -1            # no expert at all: zeros
    ids[1, 1] = -1
    ids[3] = ids[3, 0]     # the same expert three times
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = m(x, ids, w, y_dtype=torch.float32, dev_status=st)
    assert int(st.item()) == 0 and not y[0].any()
    m.check(y, x, ids, w)
    bad = ids.clone()
    bad[2, 0], bad[4, 2] = 8, -7
    y = m(x, bad, w, y_dtype=torch.float32, dev_status=st)
    assert int(st.item()) == gq.GQ_DEV_RANGE
    m.check(y, x, bad, w)
    assert not m(x, torch.full_like(ids, -1), w, y_dtype=torch.float32).any()


def test_layer_nonfinite_tokens_stay_alone():
    m = Layer(Q40, 8, 512, 192)
    x, ids, w = inputs(6, 512, 8, 2, "f32", seed=5)
    ids[:] = torch.tensor([3, 5], dtype=torch.int32)
    good = m(x, ids, w, y_dtype=torch.float32)
    x[2, 7], x[4, 100] = float("nan"), float("inf")
    y = m(x, ids, w, y_dtype=torch.float32)
    keep = [0, 1, 3, 5]
    assert torch.equal(y[keep], good[keep])
    assert not torch.isfinite(y[2]).any() and not torch.isfinite(y[4]).any()
    # and the workspace is clean afterwards
    x[2, 7], x[4, 100] = 0.5, 0.5
    m.check(m(x, ids, w, y_dtype=torch.float32), x, ids, w)


def test_layer_workspace_serves_other_sizes_and_guards_hold():
    a, b = Layer(Q40, 8, 512, 192), Layer(Q40, 4, 64, 64)
    xa, ia, wa = inputs(9, 512, 8, 3, "f16", seed=1)
    xb, ib, wb = inputs(2, 64, 4, 2, "f16", seed=2)
    need = gq.gq_moe_workspace_bytes(gq.GQ_FMT_Q4_0, 512, 192, 9, 3)
    buf = torch.zeros(need + 512, dtype=torch.uint8, device="cuda")
    buf[need:] = 0xA5
    ws = buf[:need]
    ybuf = torch.full((11, 512), 7.0, device="cuda")
    for _ in range(2):
        a(xa, ia, wa, out=ybuf[1:10], y_dtype=torch.float32, workspace=ws)
        yb = b(xb, ib, wb, y_dtype=torch.float32, workspace=ws)
        a.check(ybuf[1:10], xa, ia, wa)
        b.check(yb, xb, ib, wb)
    assert bool((buf[need:] == 0xA5).all())
    assert bool((ybuf[0] == 7).all()) and bool((ybuf[10] == 7).all())


# ------------------------------------------------------------------- router
@pytest.mark.parametrize("T,H,E,k,xt,wt", [
    (1, 8, 1, 1, "f32", "f32"), (1, 2048, 64, 6, "bf16", "bf16"), (3, 40, 7, 7, "f16", "f32"),
    (9, 4096, 256, 8, "f16", "bf16"), (17, 712, 33, 16, "f32", "f16"), (100, 128, 1000, 4, "bf16", "f16"),
])
@pytest.mark.parametrize("mode", ["softmax", "norm", "sigmoid", "sigmoid_bias"])
def test_route(T, H, E, k, xt, wt, mode):
    g = torch.Generator().manual_seed(T * H)
    x = torch.randn(T, H, generator=g).to(DT[xt])
    Wr = (torch.randn(E, H, generator=g) / H ** 0.5).to(DT[wt])
    bias = 0.2 * torch.randn(E, generator=g) if mode == "sigmoid_bias" else None
    sig, norm = mode.startswith("sigmoid"), mode != "softmax"
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    flags = (gq.GQ_ROUTE_SIGMOID if sig else 0) | (gq.GQ_ROUTE_NORM if norm else 0)
    ids, w = gq.gq_moe_route(x.cuda(), Wr.cuda(), k, bias=None if bias is None else bias.cuda(),
                             scale=1.5, flags=flags, dev_status=st)
    want, ww = moe_ref.route(x.double().numpy(), Wr.double().numpy(), k,
                             None if bias is None else bias.double().numpy(), sig, norm, 1.5)
    assert int(st.item()) == 0
    assert np.array_equal(ids.cpu().numpy(), want)
    # exponentials (2 steps), the fp32 rounding of z - max (its size times half a step), a sum of at
    # most 1024 terms in 32 + 5 additions, the quotient and the product
    z = x.double().numpy() @ Wr.double().numpy().T
    spread = np.max(z.max(1) - z.min(1)) if not sig else 0.0
    assert np.all(np.abs(w.double().cpu().numpy() - ww) <= (spread + 45) * 2.0 ** -24 * ww)


def test_route_ties_take_the_lowest_index():
    x = torch.ones(2, 16, device="cuda")
    Wr = torch.zeros(70, 16, device="cuda")
    Wr[40:44] = 1.0
    ids, w = gq.gq_moe_route(x, Wr, 6, flags=gq.GQ_ROUTE_NORM)
    assert ids.tolist() == [[40, 41, 42, 43, 0, 1]] * 2
    Wr[5] = -0.0
    Wr[3] = 0.0
    ids, _ = gq.gq_moe_route(x, -Wr, 4)  # zeros of both signs are equal
    assert ids.tolist() == [[0, 1, 2, 3]] * 2


def test_route_nonfinite_tokens():
    x = torch.randn(10, 64, device="cuda")
    Wr = torch.randn(16, 64, device="cuda")
    good = gq.gq_moe_route(x, Wr, 3)
    x[4, 5], x[9, 0] = float("nan"), float("inf")
    for flags in (0, gq.GQ_ROUTE_SIGMOID):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        ids, w = gq.gq_moe_route(x, Wr, 3, flags=flags, dev_status=st)
        assert ids[4].tolist() == [-1] * 3 and not w[4].any()
        assert int(st.item()) == gq.GQ_DEV_NONFINITE
        if not flags:  # a sigmoid of an infinity is finite
            assert ids[9].tolist() == [-1] * 3
            keep = [0, 1, 2, 3, 5, 6, 7, 8]
            assert torch.equal(ids[keep], good[0][keep]) and torch.equal(w[keep], good[1][keep])


def test_route_then_layer_chained_captured_and_on_another_stream():
    m = Layer(Q40, 16, 256, 704)
    g = torch.Generator().manual_seed(2)
    Wr = torch.randn(16, 256, generator=g).cuda()
    x = torch.randn(6, 256, generator=g).half().cuda()

    def step():
        ids, w = gq.gq_moe_route(x, Wr, 4, flags=gq.GQ_ROUTE_NORM)
        return m(x, ids, w, flags=gq.GQ_GEMV_PDL, y_dtype=torch.float32), ids, w

    y, ids, w = step()
    m.check(y, x, ids, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y2, _, _ = step()
    s.synchronize()
    assert torch.equal(y, y2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y3, ids3, w3 = step()
        y4 = m(y3.half(), ids3, w3, flags=gq.GQ_GEMV_PDL, y_dtype=torch.float32)
    for seed in (3, 4):
        x.copy_(torch.randn(6, 256, generator=torch.Generator().manual_seed(seed)).half())
        graph.replay()
        y5, ids5, w5 = step()
        torch.cuda.synchronize()
        assert torch.equal(y3, y5) and torch.equal(ids3, ids5) and torch.equal(w3, w5)
        m.check(y3, x, ids3, w3)
        m.check(y4, y3.half(), ids3, w3)


def test_layer_matches_the_grouped_products():
    # the same experts through gq_gemv_*_tiled, one token: the layer's own path beside the framework's
    m = Layer(Q40, 4, 64, 64)
    x, _, _ = inputs(1, 64, 4, 1, "f16", seed=8)
    one = lambda T, R, K, e: T.view(4, -1)[e].contiguous()  # noqa: E731
    for e in range(4):
        ids = torch.tensor([[e]], dtype=torch.int32, device="cuda")
        y = m(x, ids, torch.ones(1, 1, device="cuda"), y_dtype=torch.float32)
        a = gq.gq_gemv_q4_0_tiled(one(m.gate, 64, 64, e), 64, 64, x, y_dtype=torch.float32)
        b = gq.gq_gemv_q4_0_tiled(one(m.up, 64, 64, e), 64, 64, x, y_dtype=torch.float32)
        h = (torch.nn.functional.silu(a) * b).half()
        z = gq.gq_gemv_q4_0_tiled(one(m.down, 64, 64, e), 64, 64, h, y_dtype=torch.float32)
        scale = float(np.abs(m.d[0][e]).sum(1).max() * h.abs().max())
        assert float((y - z).abs().max()) <= (2.0 ** -11 + 1e-4) * scale  # h rounded to fp16 in one of the two
