"""The self-tests of the newer kernels' bounded waits refuse what they cannot
run before any launch (fake addresses are never touched)."""
import bit_gemv_q4_b200 as gq

INVALID, SHAPE, ALIGN, WORKSPACE = 1, 2, 3, 9
A = 0x10000000  # aligned fake device address


def test_moe_selftest_refusals():
    ok = dict(g=A, u=A, d=A, E=4, H=128, I=64, x=A, T=3, ids=A, w=A, k=2, y=A, ws=A, wsb=1 << 24, st=A)

    def call(**kw):
        a = dict(ok, **kw)
        return gq.lib.gq_selftest_moe_timeout(a["g"], a["u"], a["d"], a["E"], a["H"], a["I"], a["x"], a["T"],
                                              a["ids"], a["w"], a["k"], a["y"], a["ws"], a["wsb"], a["st"], None)

    assert call(st=None) == INVALID and call(st=A + 2) == ALIGN
    assert call(T=-1) == INVALID and call(T=65) == SHAPE and call(H=96) == SHAPE
    for n in ("g", "u", "d", "x", "ids", "w", "y"):
        assert call(**{n: None}) == INVALID and call(**{n: A + 4}) == ALIGN
    assert call(ws=None) == WORKSPACE and call(wsb=0) == WORKSPACE and call(ws=A + 128) == ALIGN
