"""The router and the expert layer on the CPU: every refusal happens before a
launch (fake addresses are never touched)."""
import pytest
import torch

import bit_gemv_q4_b200 as gq

INVALID, SHAPE, ALIGN, DTYPE, WORKSPACE = 1, 2, 3, 4, 9
A = 0x10000000  # aligned fake device address


def test_route_refusals():
    ok = dict(x=A, xt=1, T=4, H=64, w=A, wt=2, E=8, bias=None, k=2, scale=1.0, ids=A, weights=A, ws=A,
              wsb=1 << 20, flags=0, st=None)

    def call(**kw):
        a = dict(ok, **kw)
        return gq.lib.gq_moe_route(a["x"], a["xt"], a["T"], a["H"], a["w"], a["wt"], a["E"], a["bias"],
                                   a["k"], a["scale"], a["ids"], a["weights"], a["ws"], a["wsb"],
                                   a["flags"], a["st"], None)

    for n in ("T", "H", "E", "k"):
        assert call(**{n: -1}) == INVALID
    assert call(xt=3) == DTYPE and call(wt=-1) == DTYPE
    assert call(flags=8) == INVALID
    assert call(bias=A) == INVALID                       # a bias needs sigmoid scores
    assert call(bias=A + 4, flags=gq.GQ_ROUTE_SIGMOID) == ALIGN
    assert call(k=9) == SHAPE and call(E=1025) == SHAPE and call(k=17, E=64) == SHAPE
    assert call(H=60) == SHAPE and call(T=65537) == SHAPE and call(H=1 << 25) == SHAPE
    for n in ("x", "w", "ids", "weights"):
        assert call(**{n: None}) == INVALID
        assert call(**{n: A + 8}) == ALIGN
    assert call(st=A + 2) == ALIGN
    need = gq.gq_moe_route_workspace_bytes(4, 8)
    assert call(ws=None) == WORKSPACE and call(wsb=need - 1) == WORKSPACE and call(ws=A + 16) == ALIGN
    assert call(T=0) == 0 and call(k=0) == 0
    assert gq.gq_moe_route_workspace_bytes(0, 8) == 0 and gq.gq_moe_route_workspace_bytes(4, 1025) == 0


@pytest.mark.parametrize("name,fmt,step", [("gq_moe_q4_0_tiled", 0, 64), ("gq_moe_ksb_tiled", 1, 256)])
def test_layer_refusals(name, fmt, step):
    ok = dict(g=A, u=A, d=A, E=4, H=2 * step, I=step, x=A, xt=1, T=3, ids=A, w=A, k=2, y=A, yt=1, ws=A,
              wsb=1 << 24, flags=0, st=None)

    def call(**kw):
        a = dict(ok, **kw)
        return getattr(gq.lib, name)(a["g"], a["u"], a["d"], a["E"], a["H"], a["I"], a["x"], a["xt"],
                                     a["T"], a["ids"], a["w"], a["k"], a["y"], a["yt"], a["ws"], a["wsb"],
                                     a["flags"], a["st"], None)

    for n in ("E", "H", "I", "T", "k"):
        assert call(**{n: -1}) == INVALID
    assert call(xt=7) == DTYPE and call(yt=7) == DTYPE
    assert call(flags=2) == INVALID
    assert call(T=65) == SHAPE and call(k=17) == SHAPE and call(E=1025) == SHAPE
    assert call(H=step // 2) == SHAPE and call(I=3 * step // 2) == SHAPE
    assert call(H=16384 + step) == SHAPE and call(I=16384 + step) == SHAPE
    for n in ("g", "u", "d", "x", "ids", "w", "y"):
        assert call(**{n: None}) == INVALID
        assert call(**{n: A + 4}) == ALIGN
    assert call(st=A + 1) == ALIGN
    need = gq.gq_moe_workspace_bytes(fmt, 2 * step, step, 3, 2)
    assert need > 0
    assert call(ws=None) == WORKSPACE and call(wsb=need - 1) == WORKSPACE and call(ws=A + 128) == ALIGN
    assert call(T=0) == 0 and call(H=0) == 0
    assert gq.gq_moe_workspace_bytes(fmt, step // 2, step, 3, 2) == 0
    assert gq.gq_moe_workspace_bytes(fmt, step, step, 65, 2) == 0
    assert gq.gq_moe_workspace_bytes(9, step, step, 1, 2) == 0


def test_binding_refusals():
    x = torch.zeros(2, 64)
    with pytest.raises(ValueError):
        gq.gq_moe_route(x, torch.zeros(8, 32), 2)
    with pytest.raises(TypeError):
        gq.gq_moe_route(x.double(), torch.zeros(8, 64), 2)
    ids, w = torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, 1)
    big = torch.zeros(4 * 64 * 36, dtype=torch.uint8)
    with pytest.raises(TypeError):
        gq.gq_moe_q4_0_tiled(big, big, big, 4, 64, x, ids.long(), w)
    with pytest.raises(ValueError):  # storage of too few experts
        gq.gq_moe_q4_0_tiled(big[:-1], big, big, 4, 64, x, ids, w)
    with pytest.raises(ValueError):
        gq.gq_moe_q4_0_tiled(big, big, big, 4, 64, x, ids[:1], w)
