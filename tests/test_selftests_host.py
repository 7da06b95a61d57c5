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


def test_gemm_selftest_refusals():
    ok = dict(W=A, ws=A, M=256, K=128, X=A, xs=A, B=100, Y=A, work=A, wb=1 << 26, st=A)

    def call(**kw):
        a = dict(ok, **kw)
        return gq.lib.gq_selftest_gemm_fp8_timeout(a["W"], a["ws"], a["M"], a["K"], a["X"], a["xs"], a["B"],
                                                   a["Y"], a["work"], a["wb"], a["st"], None)

    assert call(st=None) == INVALID and call(st=A + 2) == ALIGN
    assert call(B=4) == SHAPE  # a kernel that waits for nothing
    assert call(M=-1) == INVALID and call(K=120) == SHAPE
    for n in ("W", "ws", "X", "xs", "Y"):
        assert call(**{n: None}) == INVALID and call(**{n: A + 4}) == ALIGN
    assert call(K=4096, work=None) == WORKSPACE
