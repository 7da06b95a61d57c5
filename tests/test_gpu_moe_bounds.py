"""The expert layer against a 64-bit form where a loose bound would hide a
mistake: activations of very small size, whose scaling by powers of two has to
bring every bit back, and fp32 activations with 16-bit outputs.  No allowance is
above a small part of a token's largest output, so an output of zeros fails."""
import numpy as np
import pytest
import torch

import moe_ref
from gpu_helpers import KSB, Q40
from test_gpu_moe import DT, Layer, inputs

pytestmark = pytest.mark.gpu

# half of the smallest step that outputs of a type have
SMALLEST = {torch.float32: 2.0 ** -150, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}


def bound(m, x, ids, w, ytype):
    """(y, allowed error): the steps of moe_ref.layer, with the absolute terms of the type at hand.
    A token's scale is 2^114 at most, so values are cut to 2^-138 (half of it: 2^-139) at the least."""
    f32_out = ytype == torch.float32
    T, H = x.shape
    y, err = np.zeros((T, H)), np.zeros((T, H))
    for t in range(T):
        for e, wt in zip(ids[t], w[t]):
            cut = np.full(H, 2.0 ** -139)
            g, dg = moe_ref.product(m.g[0][e], m.g[1][e], x[t], cut, H, m.f32_in)
            u, du = moe_ref.product(m.u[0][e], m.u[1][e], x[t], cut, H, m.f32_in)
            s = g / (1 + np.exp(np.minimum(-g, 700.0)))
            h = s * u
            # silu's slope is below 1.1; its own roundings: 8 steps; h may be subnormal
            dh = 1.1 * dg * (np.abs(u) + du) + np.abs(s) * du + 8 * 2.0 ** -23 * np.abs(h) + 2.0 ** -149 + 2.0 ** -139
            if not f32_out:  # h as one fp16 value: half a step
                dh = dh + 2.0 ** -11 * (np.abs(h) + dh)
            o, do = moe_ref.product(m.d[0][e], m.d[1][e], h, dh, m.I, f32_out)
            y[t] += wt * o
            err[t] += abs(wt) * (do + 3 * 2.0 ** -23 * np.abs(o)) + 3 * 2.0 ** -150
    return y, err + torch.finfo(ytype).eps / 2 * (np.abs(y) + err) + SMALLEST[ytype]


def check(m, x, ids, w, ytype):
    m.f32_in = x.dtype == torch.float32
    y = m(x, ids, w, y_dtype=ytype).double().cpu().numpy()
    want, allow = bound(m, x.double().cpu().numpy(), ids.cpu().numpy(), w.double().cpu().numpy(), ytype)
    assert np.all(allow.max(axis=1) < 0.1 * np.abs(want).max(axis=1))
    err = np.abs(y - want)
    assert np.all(np.isfinite(y)) and np.all(err <= allow), float((err / allow).max())


@pytest.mark.parametrize("T", [1, 4])
@pytest.mark.parametrize("spread", [1e-6, 1e-12, 1e-17, 1e4])
@pytest.mark.parametrize("xt,yt", [("bf16", "f32"), ("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16")])
def test_layer_scales_of_activations(T, spread, xt, yt):
    m = Layer(Q40, 8, 512, 192)
    x, ids, w = inputs(T, 512, 8, 2, xt, seed=9, spread=spread)
    if T > 1 and spread > 1e-17:
        x[1] *= 1e-3
    check(m, x, ids, w, DT[yt])


@pytest.mark.parametrize("fmt,E,H,I,T,k", [
    (Q40, 8, 512, 192, 1, 2), (Q40, 8, 2112, 320, 5, 3), (KSB, 4, 256, 512, 9, 2), (Q40, 2, 256, 2176, 20, 2),
])
@pytest.mark.parametrize("yt", ["f16", "bf16"])
def test_layer_fp32_activations_with_16_bit_outputs(fmt, E, H, I, T, k, yt):
    m = Layer(fmt, E, H, I)
    x, ids, w = inputs(T, H, E, k, "f32", seed=T + I)
    check(m, x, ids, w, DT[yt])
