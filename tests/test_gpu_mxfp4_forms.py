"""Every kernel that the launch rules choose between, on operands whose FP32 sums
are exact whatever their order: C has to be the exact sum rounded to BF16 once.

Products of E2M1 values are multiples of 1/4; with scales of 1 and 2 a sum of K
of them stays below 2^24 of those as long as K * 36 * 4 * 4 < 2^24, with BF16
activations (integers up to 32, scales 1 and 2) as long as K * 32 * 12 * 2 does.
A lost or repeated block of K, or a part rounded to fewer bits, shows in full."""
import numpy as np
import pytest
import torch

import mxfp4_ref as ref
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32

# 256 x 256 tiles (at least 205 of them): one to four stages of 256 K values, the
# last one partly past K; edges in M and N
LARGE_TILES = [(3601, 3715, 160), (257, 26301, 288), (3700, 3841, 544), (3585, 3840, 1024)]
# fragments straight from memory, 32 rows of B a workgroup (N from 6113 on)
WIDE_STREAM = [(1, 6113, 160), (17, 6145, 2016), (40, 7001, 96), (64, 6113, 3968)]
# rings (long rows of B): 1 to 4 fragments of A, runs of unequal length
RINGS = [(1, 3201, 4128), (32, 3169, 5152), (33, 3203, 8224), (64, 3300, 4096)]
PRODUCTS = LARGE_TILES + WIDE_STREAM + RINGS + [(100, 129, 2016), (257, 300, 12320)]
# 32 rows of B, one K block a buffer and two (K from 8192 on), K in one part and in two
WIDE_STREAM_BF16A = [(1, 6113, 544), (16, 8201, 1056), (3, 6113, 8224), (16, 8200, 8160)]
# activations in LDS: stages of every remainder by the depth, with and without
# a whole round of the ring, N and K with tails
SHARED_BF16A = [(M, 2049 + 2 * s, 256 * s - 96 + 32 * (s % 3))
                for M, last in ((17, 9), (33, 13), (49, 9)) for s in range(1, last + 1)]
BF16A = WIDE_STREAM_BF16A + SHARED_BF16A + [(16, 300, 2080), (48, 65, 544)]
# row direction, four passes a workgroup (from 2^24 values on)
MANY_ROWS = [(4101, 4111), (131075, 131)]


@pytest.fixture(scope="module")
def dg():
    need_gpu()
    import fp8_block_scaled_dg_amd as m
    return m


def operand(rng, rows, K):
    """Codes, scale words and values."""
    q = rng.integers(0, 256, (rows, K // 2)).astype(np.uint8)
    byte = np.zeros((rows, -(-K // 128) * 4), dtype=np.uint8)
    byte[:, :K // 32] = rng.integers(127, 129, (rows, K // 32))
    sf = np.ascontiguousarray(byte.view("<i4").T)
    return q, sf, ref.values(q, sf)


def dev(*a):
    return [torch.from_numpy(np.ascontiguousarray(t)).cuda() for t in a]


def rounded(a, b):
    with np.errstate(invalid="ignore"):
        c = (a @ b.T).astype(np.float32)
    return torch.from_numpy(c).to(BF16).double().numpy()


def same(c, want):
    assert np.array_equal(c.double().cpu().numpy(), want, equal_nan=True)


@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_product(dg, M, N, K):
    assert K * 36 * 4 * 4 < 2 ** 24
    rng = np.random.default_rng(M + N + K)
    (qa, sa, va), (qb, sb, vb) = operand(rng, M, K), operand(rng, N, K)
    a, b, da, db = dev(qa, qb, sa, sb)
    work = dg.alloc_workspace(dg.dg_mxfp4_gemm_nt_workspace_bytes(M, N, K))
    c = torch.full((M, N), float("nan"), dtype=BF16, device="cuda")
    for ws in (work, None):
        c.fill_(float("nan"))
        dg.dg_mxfp4_gemm_nt(c, a, b, da, db, workspace=ws)
        same(c, rounded(va, vb))
    # a NaN scale in a row of A and in a row of B; scale bytes past K are ignored
    (m, n), (i, j) = rng.integers(0, (M, N)), rng.integers(0, K // 32, 2)
    for s, row, blk in ((sa, m, i), (sb, n, j)):
        byte = s.view(np.uint8).reshape(s.shape[0], -1, 4)
        byte[blk // 4, row, blk % 4] = 255
        if K % 128:
            byte[-1, :, K // 32 % 4:] = rng.integers(0, 256, (byte.shape[1], 4 - K // 32 % 4))
    want = rounded(va, vb)
    want[m, :], want[:, n] = np.nan, np.nan
    dg.dg_mxfp4_gemm_nt(c, a, b, *dev(sa, sb), workspace=work)
    same(c, want)
    assert not work[:dg.WORKSPACE_COUNTER_BYTES].any()


@pytest.mark.parametrize("M,N,K", BF16A)
def test_product_bf16a(dg, M, N, K):
    assert K * 32 * 12 * 2 < 2 ** 24
    rng = np.random.default_rng(M + N + K)
    x = rng.integers(-32, 33, (M, K)).astype(np.float64)
    qb, sb, vb = operand(rng, N, K)
    a = torch.from_numpy(x).to(BF16).cuda()
    b, db = dev(qb, sb)
    work = dg.alloc_workspace(dg.dg_mxfp4_gemm_nt_bf16a_workspace_bytes(M, N, K))
    c = torch.full((M, N), float("nan"), dtype=BF16, device="cuda")
    for ws in (work, None):
        c.fill_(float("nan"))
        dg.dg_mxfp4_gemm_nt_bf16a(c, a, b, db, workspace=ws)
        same(c, rounded(x, vb))
    # a NaN scale; an infinity and a NaN in A: their rows alone
    n, j, k = rng.integers(0, N), rng.integers(0, K // 32), rng.integers(0, K)
    byte = sb.view(np.uint8).reshape(sb.shape[0], -1, 4)
    byte[j // 4, n, j % 4] = 255
    if K % 128:
        byte[-1, :, K // 32 % 4:] = rng.integers(0, 256, (N, 4 - K // 32 % 4))
    x[0, k] = np.inf
    if M > 1:
        x[M - 1, k] = np.nan
    want = rounded(x, vb)
    want[:, n] = np.nan
    dg.dg_mxfp4_gemm_nt_bf16a(c, torch.from_numpy(x).to(BF16).cuda(), b, *dev(sb), workspace=work)
    same(c, want)
    assert not work[:dg.WORKSPACE_COUNTER_BYTES].any()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,cols", MANY_ROWS)
def test_quantise_many_rows(dg, rows, cols, dtype):
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randn(rows, cols + 5, device="cuda", generator=g).to(dtype)
    x[::7] *= 1e-30
    x[3, 40], x[rows - 1, cols - 1] = float("inf"), float("nan")
    x = x[:, 2:cols + 2]
    q, sf = dg.to_mxfp4(x)
    want_q, want_sf = ref.quantize(x.double().cpu().numpy())
    assert np.array_equal(sf.cpu().numpy(), want_sf) and np.array_equal(q.cpu().numpy(), want_q)
