"""MXFP4 quantiser, its inverse and the MXFP4 products against plain 64-bit
numpy (mxfp4_ref.py, where the bounds are derived)."""
import numpy as np
import pytest
import torch

import mxfp4_ref as ref
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def dg():
    need_gpu()
    import fp8_block_scaled_dg_amd as m
    return m


def f64(t):
    return t.double().cpu().numpy()


def matrix(rows, cols, dtype, seed, pad=0):
    """N(0,1) with hot channels, all-zero rows and columns, tiny and huge rows,
    ties; a slice of a wider tensor when pad > 0."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, cols + pad))
    x[:, rng.random(cols + pad) < 0.02] *= 30
    x[rng.random(rows) < 0.1] = 0
    x[rng.random(rows) < 0.1] *= 1e-38
    x[rng.random(rows) < 0.1] *= 1e36
    half = rng.random(rows) < 0.2     # values on the grid's ties
    x[half] = rng.integers(-32, 33, (int(half.sum()), cols + pad)) / 4.0
    return torch.from_numpy(x.astype(np.float32)).to(dtype).cuda()[:, :cols]


def check_pair(got, x64):
    q, sf = ref.quantize(x64)
    assert np.array_equal(got[1].cpu().numpy(), sf)
    assert np.array_equal(got[0].cpu().numpy(), q)


SHAPES = [(1, 1), (1, 32), (3, 31), (32, 33), (5, 128), (129, 64), (64, 200), (100, 513), (257, 1000),
          (300, 2080), (1, 8191), (1025, 130)]


@pytest.mark.parametrize("pad", [0, 8, 13])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_quantize(dg, rows, cols, dtype, pad):
    x = matrix(rows, cols, dtype, seed=rows + cols, pad=pad)
    x64 = f64(x)
    row, col = dg.to_mxfp4(x), dg.to_mxfp4(x, transposed=True)
    check_pair(row, x64)
    check_pair(col, x64.T)
    q, sf, qt, sft = dg.to_mxfp4_both(x)
    for a, b in zip((q, sf, qt, sft), row + col):
        assert torch.equal(a, b)
    for (a, s), v in ((row, x64), (col, x64.T)):
        for out in (BF16, F32):
            back = f64(dg.from_mxfp4(a, s, v.shape[1], out))
            want = ref.values(a.cpu().numpy(), s.cpu().numpy())[:, :v.shape[1]]
            assert np.array_equal(back, want)
            assert np.array_equal(np.signbit(back), np.signbit(want))


def test_quantize_misaligned_start(dg):
    x = matrix(70, 300, BF16, seed=1)[1:, 3:260]
    check_pair(dg.to_mxfp4(x), f64(x))
    check_pair(dg.to_mxfp4(x, transposed=True), f64(x).T)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_quantize_infinities_and_nan(dg, dtype):
    x = matrix(70, 300, dtype, seed=2).contiguous()
    x[3, 40], x[64, 299], x[10, 0] = float("inf"), float("nan"), -float("inf")
    x[11, 64:96] = torch.finfo(dtype).max
    x[12, 64:96] = torch.finfo(dtype).min
    x64 = f64(x)
    q, sf, qt, sft = dg.to_mxfp4_both(x)
    check_pair((q, sf), x64)
    check_pair((qt, sft), x64.T)
    back = f64(dg.from_mxfp4(q, sf, 300, F32))
    assert np.isnan(back[3, 32:64]).all() and np.isnan(back[64, 288:]).all()
    assert np.isfinite(back[3, :32]).all()


def operand(rows, K, seed, scale=1.0):
    rng = np.random.default_rng(seed)
    q, sf = ref.quantize(rng.standard_normal((rows, K)) * scale * (1 + 20 * (rng.random(K) < 0.02)))
    return q, sf


def dev(*a):
    return [torch.from_numpy(np.ascontiguousarray(t)).cuda() for t in a]


PRODUCTS = [(1, 1, 32), (1, 128, 128), (2, 7, 96), (16, 16, 512), (17, 130, 160), (33, 257, 1056),
            (64, 300, 4096), (64, 1024, 16384), (65, 63, 64), (100, 129, 2016), (128, 256, 256),
            (200, 1000, 544), (255, 257, 288), (256, 256, 1024), (257, 515, 4128), (1000, 300, 2080),
            (513, 2049, 160), (2001, 384, 1024), (300, 1000, 2016)]


# few tiles and a long K: parts of K meet in the workspace
# (long rows of B and 16 to 64 rows of A: rings in LDS, runs of unequal length)
SPLIT_PRODUCTS = [(1, 3201, 4000), (16, 3300, 4128), (31, 3203, 4512), (48, 3201, 4064), (64, 3333, 6880),
                  (130, 7, 16384), (65, 129, 6176), (257, 300, 12320), (600, 500, 6400)]


@pytest.mark.parametrize("ws", [True, False])
@pytest.mark.parametrize("M,N,K", PRODUCTS + SPLIT_PRODUCTS)
def test_product(dg, M, N, K, ws):
    qa, sa = operand(M, K, M + K)
    qb, sb = operand(N, K, N + K + 1, 0.02)
    a, b, da, db = dev(qa, qb, sa, sb)
    work = None
    if ws:
        work = dg.alloc_workspace(dg.dg_mxfp4_gemm_nt_workspace_bytes(M, N, K))
    c = torch.full((M, N), float("nan"), dtype=BF16, device="cuda")
    dg.dg_mxfp4_gemm_nt(c, a, b, da, db, workspace=work)
    want, bound = ref.product(ref.values(qa, sa), ref.values(qb, sb))
    ref.check(f64(c), want, bound, "%dx%dx%d" % (M, N, K))
    again = dg.mxfp4_gemm_nt(a, b, da, db, workspace=work)
    assert torch.equal(again, c)
    if ws:
        assert not work[:dg.WORKSPACE_COUNTER_BYTES].any()


BF16A = [(1, 1, 32), (1, 24, 96), (2, 130, 128), (3, 257, 1056), (8, 1000, 4096), (16, 64, 160),
         (17, 300, 2048), (31, 129, 8224), (33, 512, 16384), (48, 65, 544), (49, 1023, 1024),
         (64, 384, 2080), (64, 4096, 7168)]


@pytest.mark.parametrize("ws", [True, False])
@pytest.mark.parametrize("M,N,K", BF16A)
def test_product_bf16a(dg, M, N, K, ws):
    rng = np.random.default_rng(M * N + K)
    a = torch.from_numpy(rng.standard_normal((M, K)) * (1 + 20 * (rng.random(K) < 0.02))).to(BF16).cuda()
    qb, sb = operand(N, K, N + K + 1, 0.02)
    b, db = dev(qb, sb)
    work = None
    if ws:
        work = dg.alloc_workspace(dg.dg_mxfp4_gemm_nt_bf16a_workspace_bytes(M, N, K))
    c = torch.full((M, N), float("nan"), dtype=BF16, device="cuda")
    dg.dg_mxfp4_gemm_nt_bf16a(c, a, b, db, workspace=work)
    want, bound = ref.product(f64(a), ref.values(qb, sb))
    ref.check(f64(c), want, bound, "%dx%dx%d" % (M, N, K))
    again = torch.zeros_like(c)
    dg.dg_mxfp4_gemm_nt_bf16a(again, a, b, db, workspace=work)
    assert torch.equal(again, c)
    if ws:
        assert not work[:dg.WORKSPACE_COUNTER_BYTES].any()


@pytest.mark.parametrize("M", [5, 64, 300])
def test_scale_bytes_past_k_are_ignored(dg, M):
    N, K = 200, 160                    # the second word of a row has one block
    qa, sa = operand(M, K, 1)
    qb, sb = operand(N, K, 2)
    want, bound = ref.product(ref.values(qa, sa), ref.values(qb, sb))
    for s in (sa, sb):
        s.view(np.uint8).reshape(2, -1, 4)[1, :, 1:] = [255, 254, 255]
    a, b, da, db = dev(qa, qb, sa, sb)
    ref.check(f64(dg.mxfp4_gemm_nt(a, b, da, db)), want, bound)
    if M <= dg.MXFP4_BF16A_MAX_M:
        x = torch.from_numpy(ref.values(qa, operand(M, K, 1)[1])).to(BF16).cuda()
        c = torch.empty(M, N, dtype=BF16, device="cuda")
        dg.dg_mxfp4_gemm_nt_bf16a(c, x, b, db)
        ref.check(f64(c), want, bound)


@pytest.mark.parametrize("M", [7, 300])
def test_nan_and_extreme_scales(dg, M):
    N, K = 300, 512
    qa, sa = operand(M, K, 3)
    qb, sb = operand(N, K, 4)
    byte_a, byte_b = (s.view(np.uint8).reshape(4, -1, 4) for s in (sa, sb))
    byte_a[1, 3, 2] = 255              # row 3 of C is NaN
    byte_b[2, 100, 0] = 255            # column 100 of C is NaN
    byte_b[:, 5, :] = 10               # a tiny row of B: sums far below 1, normal
    byte_a[:, 1, :] = 220              # a huge row of A
    a, b, da, db = dev(qa, qb, sa, sb)
    va, vb = ref.values(qa, sa), ref.values(qb, sb)
    want, bound = ref.product(np.nan_to_num(va), np.nan_to_num(vb))
    want[3, :], want[:, 100] = np.nan, np.nan
    ref.check(f64(dg.mxfp4_gemm_nt(a, b, da, db)), want, bound)


def test_products_and_quantiser_in_a_graph_and_on_a_stream(dg):
    M, N, K = 48, 520, 4096
    x = matrix(M, K, BF16, 5).contiguous()
    w = (torch.randn(N, K, device="cuda") * 0.02).to(BF16)
    ws = dg.alloc_workspace(max(dg.dg_mxfp4_gemm_nt_workspace_bytes(M, N, K),
                                dg.dg_mxfp4_gemm_nt_bf16a_workspace_bytes(M, N, K)))
    qs = [torch.empty(s, dtype=d, device="cuda") for s, d in
          zip(dg.mxfp4_shapes(M, K) + dg.mxfp4_shapes(N, K), (torch.uint8, torch.int32) * 2)]
    c, d = (torch.empty(M, N, dtype=BF16, device="cuda") for _ in range(2))

    def step():
        dg.dg_quantize_mxfp4(x, qs[0], qs[1])
        dg.dg_quantize_mxfp4(w, qs[2], qs[3])
        dg.dg_mxfp4_gemm_nt(c, qs[0], qs[2], qs[1], qs[3], workspace=ws)
        dg.dg_mxfp4_gemm_nt_bf16a(d, x, qs[2], qs[3], workspace=ws)

    step()
    torch.cuda.synchronize()
    want = c.clone(), d.clone()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            step()
    for _ in range(3):
        c.zero_(), d.zero_(), qs[0].zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(c, want[0]) and torch.equal(d, want[1])
        c.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            step()                      # eager, on another stream than the default
        side.synchronize()
        assert torch.equal(c, want[0]) and torch.equal(d, want[1])


def test_linear_training_step_gradients(dg):
    """y, dx, dw of a linear layer with every operand quantised along its own
    contraction axis equal the 64-bit formula on the quantised operands, and
    dx, dw are the derivatives of that product (it is bilinear: differences
    of its plain form are exact up to rounding)."""
    M, N, K = 77, 160, 224
    rng = np.random.default_rng(9)
    x, w, dy = (torch.from_numpy(rng.standard_normal(s)).to(BF16).cuda()
                for s in ((M, K), (N, K), (M, N)))
    qx, qw, qd = dg.to_mxfp4_both(x), dg.to_mxfp4_both(w), dg.to_mxfp4_both(dy)
    y = dg.mxfp4_gemm_nt(qx[0], qw[0], qx[1], qw[1])
    dx = dg.mxfp4_gemm_nt(qd[0], qw[2], qd[1], qw[3])
    dw = dg.mxfp4_gemm_nt(qd[2], qx[2], qd[3], qx[3])

    def v(q, sf, cols):
        return ref.values(q.cpu().numpy(), sf.cpu().numpy())[:, :cols]
    X, W = v(*qx[:2], K), v(*qw[:2], K)
    D, WT = v(*qd[:2], N), v(*qw[2:], N)
    DT, XT = v(*qd[2:], M), v(*qx[2:], M)
    ref.check(f64(y), *ref.product(X, W))
    ref.check(f64(dx), *ref.product(D, WT))
    ref.check(f64(dw), *ref.product(DT, XT))
    # differences: loss(x, w) = sum(D . (x w^T)), along random directions
    vx, vw = rng.standard_normal((M, K)), rng.standard_normal((N, K))
    loss = lambda a, b, d: float(np.sum(d * (a @ b.T)))
    h = 0.5
    diff_x = (loss(X + h * vx, WT.T, D) - loss(X - h * vx, WT.T, D)) / (2 * h)
    diff_w = (loss(XT.T, W + h * vw, DT.T) - loss(XT.T, W - h * vw, DT.T)) / (2 * h)
    for got, direction, diff, (exact, bound) in ((dx, vx, diff_x, ref.product(D, WT)),
                                                 (dw, vw, diff_w, ref.product(DT, XT))):
        room = np.sum(np.abs(direction) * (2.0 ** -8 * np.abs(exact) + (1 + 2.0 ** -8) * bound))
        assert abs(np.sum(f64(got) * direction) - diff) <= room + 1e-9 * abs(diff)
