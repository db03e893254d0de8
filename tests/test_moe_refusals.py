"""Routing, layout, dispatch, combine and 8-bit SwiGLU: bad arguments are
rejected on the host, nothing is enqueued, no GPU needed."""
import ctypes

import pytest

P = ctypes.c_void_p(0x10000)
P1 = ctypes.c_void_p(0x10001)
P2 = ctypes.c_void_p(0x10002)
P4 = ctypes.c_void_p(0x10004)
FAR = ctypes.c_void_p(0x10000 + (1 << 40))


@pytest.fixture(scope="module")
def dg():
    import fp8_block_scaled_dg_amd as m
    return m


def test_route(dg):
    def f(ids=P, w=P, lg=P, dt=0, ldl=64, bias=None, sc=0, G=1, tg=1, best=1, T=4, E=64, k=8):
        return dg.lib.dg_moe_route(ids, w, lg, dt, ldl, bias, sc, G, tg, best, 1, 1.0, T, E, k, None)
    assert f(ids=None) == f(w=None) == f(lg=None) == 1
    assert f(dt=2) == f(dt=-1) == f(sc=2) == f(best=0) == f(best=3) == 3
    assert f(T=0) == f(T=-1) == f(T=(1 << 25) + 1) == f(E=0) == f(E=1025, ldl=1025) == 2
    assert f(k=0) == f(k=17) == f(E=4, k=5) == f(ldl=63) == f(ldl=1 << 61) == 2
    assert f(G=0) == f(G=65, E=65, ldl=65) == f(G=3) == f(tg=0) == f(G=4, tg=5) == 2
    assert f(G=64, tg=2, best=2) == 2           # one expert a group
    assert f(ids=P1) == f(w=P2) == f(lg=P2) == f(lg=P1, dt=1) == f(bias=P1) == 4


def test_route_backward(dg):
    def f(d=P, ldd=64, dw=P, ids=P, lg=P, dt=0, ldl=64, sc=0, T=4, E=64, k=8):
        return dg.lib.dg_moe_route_backward(d, ldd, dw, ids, lg, dt, ldl, sc, 1, 1.0, T, E, k, None)
    assert f(d=None) == f(dw=None) == f(ids=None) == f(lg=None) == 1
    assert f(dt=2) == f(sc=-1) == 3
    assert f(ldd=63) == f(ldl=63) == f(T=0) == f(k=0) == f(E=1025, ldl=1025, ldd=1025) == 2
    assert f(d=P2) == f(d=P1, dt=1) == f(dw=P1) == 4


def test_plan(dg):
    def f(rows=P, pairs=P, mi=P, off=P, cnt=P, ids=P, T=64, E=8, k=2, M=None, ws=P, n=1 << 20):
        M = dg.dg_moe_plan_rows(T, E, k) if M is None else M
        return dg.lib.dg_moe_plan(rows, pairs, mi, off, cnt, ids, T, E, k, M, ws, n, None)
    for name in ("rows", "pairs", "mi", "off", "cnt", "ids"):
        assert f(**{name: None}) == 1, name
    assert dg.dg_moe_plan_rows(64, 8, 2) == 128 * (8 + 120 // 128)
    assert dg.dg_moe_plan_rows(1, 8, 2) == 256 and dg.dg_moe_plan_rows(1000, 1, 1) == 1024
    assert dg.dg_moe_plan_rows(0, 8, 2) == dg.dg_moe_plan_rows(1, 8, 9) == 0
    assert dg.dg_moe_plan_rows((1 << 27) + 1, 8, 1) == dg.dg_moe_plan_rows(1 << 60, 8, 8) == 0
    assert f(M=896) == f(M=1025) == f(M=(1 << 30) + 128) == 2
    assert f(T=0, M=128) == f(E=0, M=1024) == f(k=9, M=4096) == f(k=17, E=32, M=8192) == 2
    need = dg.dg_moe_plan_workspace_bytes(65536, 256, 8)
    assert need > 0 == dg.dg_moe_plan_workspace_bytes(1, 256, 8)
    assert f(T=65536, E=256, k=8, ws=None, n=0) == f(T=65536, E=256, k=8, n=need - 1) == 5
    assert f(off=P4) == f(ids=P1) == f(ws=P4) == 4


def test_dispatch(dg):
    def f(a=P, sa=P, x=P, dt=1, ldx=256, rows=P, pairs=P, w=None, T=4, k=2, M=256, H=256, ws=None, n=0):
        return dg.lib.dg_moe_dispatch_fp8(a, sa, x, dt, ldx, rows, pairs, w, T, k, M, H, ws, n, None)
    for name in ("a", "sa", "x", "rows", "pairs"):
        assert f(**{name: None}) == 1, name
    assert f(dt=2) == 3
    assert f(T=0) == f(k=0) == f(k=17) == f(M=0) == f(M=200) == f(H=0) == f(H=192) == f(ldx=255) == 2
    assert f(T=(1 << 23) + 1) == f(M=(1 << 27) + 128) == f(T=1 << 23, H=4096, ldx=4096) == f(ldx=1 << 61) == 2
    assert f(a=P4) == f(sa=P1) == f(x=P1) == f(x=P2, dt=0) == f(w=P2) == f(pairs=P1) == 4
    need = dg.dg_moe_dispatch_fp8_workspace_bytes(8192, 8, 7168)
    assert need == 8192 * 56 * 4 and dg.dg_moe_dispatch_fp8_workspace_bytes(8192, 8, 7168, True) == 8 * need
    assert dg.dg_moe_dispatch_fp8_workspace_bytes(1, 8, 7168) == 0
    big = dict(T=8192, k=8, M=65536, H=7168, ldx=7168)
    assert f(ws=P, n=need - 1, **big) == 5 and f(ws=P4, n=need, **big) == 4


def test_combine(dg):
    def f(y=P, c=P, rows=P, w=None, res=None, T=4, k=2, M=256, H=256):
        return dg.lib.dg_moe_combine(y, c, rows, w, res, T, k, M, H, None)
    assert f(y=None) == f(c=None) == f(rows=None) == 1
    assert f(T=0) == f(k=17) == f(M=100) == f(H=4) == f(H=12) == f(T=1 << 26) == 2
    assert f(y=P4) == f(c=P4) == f(res=P4) == f(rows=P1) == f(w=P1) == 4


def test_combine_backward(dg):
    def f(dc=P, sdc=P, dw=P, dy=P, ld=256, c=P, rows=P, pairs=P, w=P, T=4, k=2, M=256, H=256):
        return dg.lib.dg_moe_combine_backward(dc, sdc, dw, dy, ld, c, rows, pairs, w, T, k, M, H, None, 0,
                                              None)
    assert f(dy=None) == f(rows=None) == f(pairs=None) == f(c=None) == f(sdc=None) == f(dc=None) == 1
    assert f(dc=None, sdc=None, dw=None) == 1
    assert f(ld=255) == f(H=136, ld=136) == f(M=64) == f(T=0) == 2
    assert f(dc=P4) == f(dy=P1) == f(c=P4) == f(dw=P1) == f(w=P2) == f(sdc=P2) == 4


def test_swiglu(dg):
    def f(h=P, sh=P, kept=None, sk=None, gu=P, mi=None, M=100, I=128):
        return dg.lib.dg_swiglu_fp8(h, sh, kept, sk, gu, mi, M, I, None)
    assert f(h=None) == f(sh=None) == f(gu=None) == f(kept=P) == f(sk=P) == 1
    assert f(M=0) == f(I=0) == f(I=64) == f(I=192) == f(M=(1 << 25) + 1) == 2
    assert f(mi=P, M=100) == 2                  # whole blocks of rows with m_indices
    assert f(h=P4) == f(gu=P2) == f(sh=P1) == f(mi=P1, M=128) == f(kept=P4, sk=P) == 4


def test_swiglu_backward(dg):
    def f(d=P, sd=P, h=None, sh=None, dh=P, kept=P, sk=P, mi=None, M=100, I=128):
        return dg.lib.dg_swiglu_fp8_backward(d, sd, h, sh, dh, kept, sk, mi, M, I, None)
    for name in ("d", "sd", "dh", "kept", "sk"):
        assert f(**{name: None}) == 1, name
    assert f(h=P) == f(sh=P) == 1
    assert f(M=0) == f(I=100) == f(mi=P, M=130) == 2
    assert f(d=P4) == f(dh=P4) == f(kept=P4) == f(sk=P1) == f(h=P4, sh=P) == 4


def test_transpose(dg):
    def f(qt=FAR, st=P, br=1, q=P, s=P, mi=None, M=128, C=128):
        return dg.lib.dg_transpose_fp8_blocks(qt, st, br, q, s, mi, M, C, None)
    assert f(qt=None) == f(st=None) == f(q=None) == f(s=None) == 1
    assert f(br=0) == f(br=64) == f(qt=P) == 3  # in place
    assert f(M=64) == f(M=192) == f(C=0) == f(C=130) == f(M=1 << 24, C=1 << 14) == 2
    assert f(q=P4) == f(s=P1) == f(st=P2) == f(mi=P1) == 4


def test_binding_refuses(dg):
    torch = pytest.importorskip("torch")
    i32 = torch.zeros(4, 2, dtype=torch.int32)
    f32, x = torch.zeros(4, 2), torch.zeros(4, 128)
    with pytest.raises(ValueError):
        dg.dg_moe_route(i32, f32, torch.zeros(4, 8))                # host tensors
    with pytest.raises(TypeError):
        dg.dg_moe_route(i32, f32, torch.zeros(4, 8).half())
    with pytest.raises(TypeError):
        dg.dg_moe_route_backward(f32, f32, i32, [1])
    with pytest.raises(ValueError):
        dg.dg_moe_plan(i32, i32, i32, i32, i32, i32)
    with pytest.raises(TypeError):
        dg.moe_plan([[1, 2]], 4)
    with pytest.raises(ValueError):
        dg.moe_plan(i32, 0)
    with pytest.raises(ValueError):
        dg.dg_moe_dispatch_fp8(None, None, x, i32, i32)
    with pytest.raises(TypeError):
        dg.dg_moe_combine(x, None, i32)
    with pytest.raises(TypeError):
        dg.dg_moe_combine_backward(None, None, f32, x, x, i32, i32)
    with pytest.raises(ValueError):
        dg.dg_swiglu_fp8(None, None, torch.zeros(4, 256, dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        dg.dg_swiglu_fp8_backward(None, None, x, None, None)
    with pytest.raises(ValueError):
        dg.dg_transpose_fp8_blocks(None, None, torch.zeros(128, 128, dtype=torch.uint8), None)
    with pytest.raises(KeyError):
        dg.MOE_SCORINGS["relu"]
