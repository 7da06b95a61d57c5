"""Plain 64-bit forms of the router and of the expert layer, with the error
that the kernels' arithmetic may make (no kernel code here).

The weights are the oracle's: quantized and decoded by it, scales read from the
packed bytes."""
import numpy as np

import oracle
from gpu_helpers import Q40


def experts(fmt, E, R, K, seed, std=0.05):
    """(packed bytes of the E * R x K matrix, decoded [E, R, K], scale of each weight)."""
    g = np.random.default_rng(seed)
    w = (g.standard_normal((E * R, K)) * std * np.exp(g.uniform(-1, 1, (E * R, 1)))).astype(np.float32)
    q, _ = oracle.quantize(fmt, w.ravel())
    dec = oracle.dequantize(fmt, q, E * R * K).astype(np.float64).reshape(E, R, K)
    if fmt == Q40:
        d = q.reshape(-1, 18)[:, :2].copy().view(np.float16).astype(np.float64)
        d = np.repeat(d, 32, axis=1)
    else:
        b = q.reshape(-1, 138)
        S = b[:, :2].copy().view(np.float16).astype(np.float64)
        d = np.repeat(S * b[:, 2:10].copy().view(np.int8).astype(np.float64), 32, axis=1)
    return q, dec, np.abs(d).reshape(E, R, K)


def product(W, d, x, dx, K, two_terms):
    """(W x, its possible error) for x known to dx.  The kernel adds (code - 8) * x: terms of |W| |x|
    in sum (16 d |x| more are let through, for a form that adds code * x and -8 * x).  A block of 32
    is two MMAs of 16 products on an accumulator input, the blocks' sums are added in fp32: at most
    K / 32 + 40 additions, each cut to 24 bits (a whole step, 2^-23, where the tensor core truncates).  Two fp16 terms hold 22
    bits of x: 2^-22 of it, and 2^-38 of the largest |x| where the remainder is subnormal."""
    ax = np.abs(x)
    mag = (np.abs(W) + 16 * d) @ ax
    err = (K / 32 + 40) * 2.0 ** -23 * mag + np.abs(W) @ dx
    low = 2.0 ** -38 * ax.max(initial=0.0)
    err += np.abs(W) @ ((2.0 ** -22 * ax if two_terms else 0.0) + np.full_like(ax, low))
    return W @ x, err


def layer(gate, up, down, x, ids, w, x_is_f32, y_half_step):
    """(y, allowed error) in 64 bits; gate, up, down: (decoded, scales); y_half_step: the type's
    eps / 2 (0 step for fp32 outputs is eps / 2 of fp32 itself)."""
    T, H = x.shape
    E, I = gate[0].shape[:2]
    f32_out = y_half_step < 2.0 ** -20
    y, err = np.zeros((T, H)), np.zeros((T, H))
    for t in range(T):
        for e, wt in zip(ids[t], w[t]):
            if not 0 <= e < E:
                continue
            zero = np.zeros(H)
            g, dg = product(gate[0][e], gate[1][e], x[t], zero, H, x_is_f32)
            u, du = product(up[0][e], up[1][e], x[t], zero, H, x_is_f32)
            s = g / (1 + np.exp(np.minimum(-g, 700.0)))
            h = s * u
            # silu's slope is below 1.1; its own roundings (exp, sum, quotient, product): 8 steps
            dh = 1.1 * dg * (np.abs(u) + du) + np.abs(s) * du + 8 * 2.0 ** -23 * np.abs(h)
            if not f32_out:  # h as one fp16 value: half a step
                dh = dh + 2.0 ** -11 * (np.abs(h) + dh)
            o, do = product(down[0][e], down[1][e], h, dh, I, f32_out)
            y[t] += wt * o
            err[t] += abs(wt) * (do + 2.0 ** -23 * np.abs(o) * 3)
    return y, err + y_half_step * (np.abs(y) + err) + 2.0 ** -25  # fp16 subnormal outputs: half of 2^-24


def route(x, Wr, k, bias=None, sigmoid=False, norm=False, scale=1.0):
    z = x @ Wr.T
    if sigmoid:
        s = 1 / (1 + np.exp(-z))
        key = s + bias if bias is not None else s
    else:
        s = np.exp(z - z.max(axis=1, keepdims=True))
        s = s / s.sum(axis=1, keepdims=True)
        key = z
    ids = np.argsort(-key, axis=1, kind="stable")[:, :k]
    w = np.take_along_axis(s, ids, axis=1)
    if norm:
        w = w / w.sum(axis=1, keepdims=True)
    return ids.astype(np.int32), w * scale
