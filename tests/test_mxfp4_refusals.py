"""MXFP4 and mixture-of-experts entry points: bad arguments are rejected on
the host (nothing is enqueued, no GPU needed), and the plain 64-bit forms the
GPU tests compare with agree with the formats' definitions."""
import ctypes

import numpy as np
import pytest

import mxfp4_ref as ref

P = ctypes.c_void_p(0x10000)
P1 = ctypes.c_void_p(0x10001)
P4 = ctypes.c_void_p(0x10004)


@pytest.fixture(scope="module")
def dg():
    import fp8_block_scaled_dg_amd as m
    return m


def test_quantize(dg):
    def f(q=P, sf=P, qt=None, sft=None, x=P, dtype=1, rows=64, cols=64, ldx=64):
        return dg.lib.dg_quantize_mxfp4(q, sf, qt, sft, x, dtype, rows, cols, ldx, None)
    assert f(x=None) == f(q=None, sf=None) == f(sf=None) == f(qt=P) == f(sft=P) == 1
    assert f(dtype=2) == f(dtype=-1) == 3
    assert f(rows=0) == f(cols=0) == f(rows=-1) == f(ldx=63) == 2
    assert f(rows=1 << 29) == 2 and f(cols=1 << 36, ldx=1 << 36) == 2
    assert f(q=P4) == f(sf=P1) == f(x=P1) == f(qt=P1, sft=P) == 4


def test_dequantize(dg):
    def f(out=P, dtype=1, q=P, sf=P, rows=64, cols=64):
        return dg.lib.dg_dequantize_mxfp4(out, dtype, q, sf, rows, cols, None)
    assert f(out=None) == f(q=None) == f(sf=None) == 1
    assert f(dtype=7) == 3
    assert f(rows=0) == f(cols=0) == f(rows=1 << 29, cols=129) == 2
    assert f(out=P4) == f(q=P4) == f(sf=P1) == 4


def test_product(dg):
    def f(c=P, a=P, b=P, sa=P, sb=P, M=64, N=64, K=64, ws=None, n=0):
        return dg.lib.dg_mxfp4_gemm_nt(c, a, b, sa, sb, M, N, K, ws, n, None)
    assert f(c=None) == f(a=None) == f(b=None) == f(sa=None) == f(sb=None) == 1
    assert f(M=0) == f(N=0) == f(K=0) == f(K=48) == f(K=(1 << 23) + 32) == 2
    assert f(N=1 << 29) == f(M=1 << 28, K=1024) == f(N=1 << 31) == 2
    assert f(a=P4) == f(b=P4) == f(sa=P1) == f(c=P1) == f(c=P4) == 4
    assert f(N=63, c=P1) == 4
    need = dg.dg_mxfp4_gemm_nt_workspace_bytes(16, 1024, 16384)
    assert need > dg.WORKSPACE_COUNTER_BYTES
    assert f(M=16, N=1024, K=16384, ws=P, n=need - 1) == 5
    assert f(M=16, N=1024, K=16384, ws=P4, n=need) == 4
    assert dg.dg_mxfp4_gemm_nt_workspace_bytes(0, 1, 32) == 0


def test_product_bf16a(dg):
    def f(c=P, a=P, b=P, sb=P, M=64, N=64, K=64, ws=None, n=0):
        return dg.lib.dg_mxfp4_gemm_nt_bf16a(c, a, b, sb, M, N, K, ws, n, None)
    assert f(c=None) == f(a=None) == f(b=None) == f(sb=None) == 1
    assert f(M=0) == f(M=dg.MXFP4_BF16A_MAX_M + 1) == f(N=0) == f(K=16) == f(K=80) == 2
    assert f(a=P4) == f(sb=P1) == 4
    need = dg.dg_mxfp4_gemm_nt_bf16a_workspace_bytes(16, 1024, 16384)
    assert f(M=16, N=1024, K=16384, ws=P, n=need - 1) == 5


def test_moe_layer(dg):
    def f(y=P, x=P, w13=P, w2=P, s13=P, s2=P, fmt=0, ids=P, w=P, lg=P, sc=0, T=4, E=8, k=2, H=256,
          I=128, ws=P, n=1 << 30):
        return dg.lib.dg_moe_layer(y, x, w13, w2, s13, s2, fmt, ids, w, lg, sc, T, E, k, H, I, ws,
                                   n, None)
    for name in ("y", "x", "w13", "w2", "s13", "s2", "ids", "w"):
        assert f(**{name: None}) == 1, name
    assert f(fmt=2) == f(sc=2) == 3
    assert f(T=0) == f(T=65) == f(E=0) == f(E=1025) == f(k=0) == f(k=9) == f(E=32, k=17) == 2
    assert f(H=0) == f(H=272) == f(I=16) == f(H=131104) == f(I=(1 << 20) + 32) == 2
    assert f(fmt=1, H=160) == f(fmt=1, I=160) == 2       # 128 x 128 blocks
    assert f(T=64, E=16, k=16, H=32, I=1 << 19) == 2     # hidden values of 2^31 bytes
    assert f(ws=None) == 5
    need = dg.dg_moe_layer_workspace_bytes(4, 8, 2, 256, 128)
    assert f(n=need - 1) == 5
    assert f(ws=P4) == f(x=P4) == f(w2=P4) == f(lg=P1) == f(ids=P1) == 4
    assert dg.dg_moe_layer_workspace_bytes(65, 8, 2, 256, 128) == 0
    # the serving range's workspaces
    assert dg.dg_moe_layer_workspace_bytes(64, 256, 8, 4096, 11008) <= 32 << 20


def test_binding_refuses(dg):
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        dg.dg_quantize_mxfp4(x, *map(torch.zeros, dg.mxfp4_shapes(4, 64)))   # host tensor
    with pytest.raises(TypeError):
        dg.dg_quantize_mxfp4(x.half())
    with pytest.raises(TypeError):
        dg.from_mxfp4(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(1, 4, dtype=torch.int32),
                      64, torch.float16)
    assert dg.mxfp4_shapes(5, 130) == ((5, 80), (2, 5))


def test_reference_quantiser_definition():
    x = np.array([[4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.9, -0.25, -0.3, -0.0] + [0.0] * 20])
    q, sf = ref.quantize(x)
    v = ref.values(q, sf)[0, :12]
    assert v.tolist() == [4, 0, 1, 1, 2, 2, 4, 4, 6, 0, -0.5, 0]
    assert np.signbit(v[9]) and np.signbit(v[11]) and sf.tolist() == [[127]]
    for e in (-126, -125, 0, 100, 127):
        q, sf = ref.quantize(x * 2.0 ** (e - 2))
        assert sf[0, 0] == max(e - 2, -127) + 127
    q, sf = ref.quantize(np.zeros((1, 33)))
    assert q.shape == (1, 32) and not q.any() and not sf.any()
    q, sf = ref.quantize(np.array([[1.0] * 32 + [np.inf] + [2.0] * 31]))
    assert sf[0, 0] == (125 | 255 << 8) and not q[0, 16:].any()
    below = np.nextafter(np.float32(8), np.float32(0)).astype(np.float64)
    assert ref.quantize(np.full((1, 32), below))[1][0, 0] == 127


def test_reference_routing():
    l = np.array([[0, 2, 2, -np.inf], [-np.inf] * 4, [np.nan, 1, -200, -300]], dtype=np.float32)
    ids, w = ref.route(l, 2, "softmax")
    assert ids.tolist() == [[1, 2], [-1, -1], [1, 2]]
    assert w[0].tolist() == [0.5, 0.5] and not w[1].any()
    ids, w = ref.route(l[2:, 2:], 2, "sigmoid")
    assert np.allclose(w, [[1, np.exp(-100)]], rtol=1e-12)
