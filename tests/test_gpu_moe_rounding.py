"""16-bit outputs of the expert layer are rounded once: hardly any differs from
the 64-bit result rounded to the type.

How many may.  An output is rounded the other way where its error before the
rounding is more than its distance to the middle between two values, which lies
evenly in 0 .. half a step: a share of 2 E|error| / step.  With the activation
between the products held to 22 bits and sums in 32 bits the error is some 2^-21
of a typical |y|.  Steps of fp16 are 2^-11 .. 2^-10 of |y|, in the mean over y's
bell about five times less (small outputs have small steps): 2 * 2^-21 * 5 *
2^11, about 1 %, and an eighth of it for bf16.  Twice that is let through.  (One
rounding of the activation to 11 bits makes it some 30 % and 4 %.)"""
import pytest
import torch

import moe_ref
from gpu_helpers import KSB, Q40
from test_gpu_moe import DT, Layer, inputs

pytestmark = pytest.mark.gpu

SHARE = {"f16": 0.02, "bf16": 0.0025}


@pytest.mark.parametrize("fmt,E,H,I,T,k", [
    (Q40, 8, 2048, 704, 1, 2),       # one token, all slots in one row
    (Q40, 2, 2048, 16384, 1, 1),
    (KSB, 4, 2048, 512, 3, 2),
    (Q40, 4, 512, 704, 33, 2),       # experts of many tokens
])
@pytest.mark.parametrize("xt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("yt", ["f16", "bf16"])
def test_layer_rounds_16_bit_outputs_once(fmt, E, H, I, T, k, xt, yt):
    m = Layer(fmt, E, H, I)
    x, ids, w = inputs(T, H, E, k, xt, seed=T + I)
    y = m(x, ids, w, y_dtype=DT[yt]).cpu()
    want, _ = moe_ref.layer(m.g, m.u, m.d, x.double().cpu().numpy(), ids.cpu().numpy(), w.double().cpu().numpy(),
                            xt == "f32", 2.0 ** -24)
    want = torch.from_numpy(want).to(DT[yt])
    assert float((y != want).double().mean()) <= SHARE[yt]
