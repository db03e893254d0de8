"""The 8-bit SwiGLU, its checkpoint, its gradient and the transposed operands.
What is quantised straight from an input is compared bit for bit with the
oracle's quantiser; what is computed in FP32 first, within the bounds of
moe_ref.py."""
import numpy as np
import pytest
import torch

import moe_ref as ref
from gpu_util import dev, need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dg():
    need_gpu()
    import fp8_block_scaled_dg_amd as m
    return m


def spoiled(M, C):
    return (torch.full((M, C), 0x7F, dtype=torch.uint8, device="cuda"),
            torch.full((C // 128, M), -3.0, device="cuda"))


def rows_of(rng, M, grouped):
    """m_indices (None: all rows real) and what each row is: real, fill, untouched."""
    if not grouped:
        return None, np.ones(M, bool), np.zeros(M, bool)
    mi = np.full(M, -1)
    for b in range(M // 128):
        n = rng.choice([0, 1, 31, 33, 127, 128])
        mi[128 * b:128 * b + n] = b
    real, used = mi >= 0, ref.blocks_used(mi)
    return dev(mi.astype(np.int32)), real, used & ~real


def untouched(q, s, real, fill):
    q, s = q.cpu().numpy(), s.cpu().numpy()
    assert not q[fill].any() and not s[:, fill].any()
    rest = ~real & ~fill
    assert (q[rest] == 0x7F).all() and (s[:, rest] == -3).all()
    return q[real], np.ascontiguousarray(s[:, real])


# M, I, grouped
SHAPES = [(1, 128, False), (3, 512, False), (37, 640, False), (128, 128, True), (384, 1408, True), (130, 4224, False),
          (1280, 256, True), (64, 11008, False)]


@pytest.mark.parametrize("M,I,grouped", SHAPES)
def test_forward_and_backward(dg, orc, M, I, grouped):
    rng = np.random.default_rng(M + I)
    mi, real, fill = rows_of(rng, M, grouped)
    gu = dev((rng.standard_normal((M, 2 * I)) * 4).astype(np.float32)).to(torch.bfloat16)
    gu[0, :256] = 0
    gu[M - 1, -6:] = torch.tensor([-90.0, 1e30, 90.0, -2.0, -0.0, 3.0], device="cuda").to(torch.bfloat16)
    out = dev(~real)
    gu[out] = float("nan")                        # what is in rows that are not real has no part in it
    h, sh = spoiled(M, I)
    dg.dg_swiglu_fp8(h, sh, gu, m_indices=mi)
    h1, sh1 = spoiled(M, I)
    kept, skept = spoiled(M, 2 * I)
    dg.dg_swiglu_fp8(h1, sh1, gu, kept, skept, m_indices=mi)
    assert torch.equal(h, h1) and torch.equal(sh, sh1)
    x = gu.double().cpu().numpy()[real]
    if not len(x):
        return
    want, err = ref.swiglu(x[:, 0::2], x[:, 1::2])
    ref.check_quantised(*untouched(h, sh, real, fill), want, err)
    qk, sk = untouched(kept, skept, real, fill)
    oq, os_ = orc.quantize(x.astype(np.float32), 1)
    assert np.array_equal(qk, oq) and np.array_equal(sk, os_)

    dh = dev((rng.standard_normal((M, I)) * 1e-2).astype(np.float32)).to(torch.bfloat16)
    dh[out] = float("nan")
    d, sd = spoiled(M, 2 * I)
    dg.dg_swiglu_fp8_backward(d, sd, dh, kept, skept, m_indices=mi)
    d1, sd1 = spoiled(M, 2 * I)
    h2, sh2 = spoiled(M, I)
    dg.dg_swiglu_fp8_backward(d1, sd1, dh, kept, skept, h2, sh2, m_indices=mi)
    assert torch.equal(d, d1) and torch.equal(sd, sd1)
    k1, sk1 = kept.clone(), skept.clone()         # in the checkpoint's place
    dg.dg_swiglu_fp8_backward(k1, sk1, dh, k1, sk1, m_indices=mi)
    assert torch.equal(d, k1) and torch.equal(sd, sk1)
    v = ref.values(qk, sk)                        # the checkpoint's values
    y = dh.double().cpu().numpy()[real]
    a, b, ea, eb = ref.swiglu_gradient(v[:, 0::2], v[:, 1::2], y)
    ref.check_quantised(*untouched(d, sd, real, fill), np.stack((a, b), -1).reshape(-1, 2 * I),
                        np.stack((ea, eb), -1).reshape(-1, 2 * I))
    ref.check_quantised(*untouched(h2, sh2, real, fill), *ref.swiglu(v[:, 0::2], v[:, 1::2]))


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("M,C,grouped", [(128, 128, False), (256, 384, False), (1280, 256, True), (384, 1408, True)])
def test_transpose(dg, orc, M, C, grouped, block_rows):
    rng = np.random.default_rng(M + C)
    mi, real, fill = rows_of(rng, M, grouped)
    x = rng.standard_normal((M, C)).astype(np.float32) * np.exp(rng.standard_normal((M, 1)) * 2).astype(np.float32)
    x[:, 5] = 0
    x[1] = 0
    q, s = orc.quantize(x, 1)
    q[fill], s[:, fill] = 0, 0
    used = real | fill
    q[~used], s[:, ~used] = 0x7F, np.nan
    qt = torch.full((C, M), 0x55, dtype=torch.uint8, device="cuda")
    st = torch.full((M // 128, C if block_rows == 1 else C // 128), -3.0, device="cuda")
    dg.dg_transpose_fp8_blocks(qt, st, dev(q), dev(s), block_rows=block_rows, m_indices=mi)
    qt, st = qt.cpu().numpy(), st.cpu().numpy()
    blocks = used.reshape(-1, 128)[:, 0]
    assert (qt[:, ~used] == 0x55).all() and (st[~blocks] == -3).all()
    if used.any():
        v = ref.values(q[used], s[:, used]).astype(np.float32)
        want, ws = orc.quantize(np.ascontiguousarray(v.T), block_rows)
        assert np.array_equal(qt[:, used], want) and np.array_equal(st[blocks], ws)


def test_past_32_bits(dg, orc):
    """Rows of gate/up, of the checkpoint and of a transposed operand that start
    past 4 GiB; all but the last block are without an expert."""
    M, I = 1 << 18, 8448
    mi = torch.full((M,), -1, dtype=torch.int32, device="cuda")
    mi[-128:-100] = 0
    real = slice(M - 128, M - 100)
    gu = torch.empty(M, 2 * I, dtype=torch.bfloat16, device="cuda")
    gu[real] = torch.randn(28, 2 * I, device="cuda").to(torch.bfloat16)
    h, sh = torch.empty(M, I, dtype=torch.uint8, device="cuda"), torch.empty(I // 128, M, device="cuda")
    kept, skept = torch.empty(M, 2 * I, dtype=torch.uint8, device="cuda"), torch.empty(I // 64, M, device="cuda")
    dg.dg_swiglu_fp8(h, sh, gu, kept, skept, m_indices=mi)
    oq, os_ = orc.quantize(gu[real].float().cpu().numpy(), 1)
    assert np.array_equal(kept[real].cpu().numpy(), oq) and np.array_equal(skept[:, real].cpu().numpy(), os_)
    dh = torch.empty(M, I, dtype=torch.bfloat16, device="cuda")
    dh[real] = torch.randn(28, I, device="cuda").to(torch.bfloat16)
    d, sd = torch.empty_like(kept), torch.empty_like(skept)
    dg.dg_swiglu_fp8_backward(d, sd, dh, kept, skept, m_indices=mi)
    v, y = ref.values(oq, os_), dh[real].double().cpu().numpy()
    a, b, ea, eb = ref.swiglu_gradient(v[:, 0::2], v[:, 1::2], y)
    ref.check_quantised(d[real].cpu().numpy(), sd[:, real].cpu().numpy(), np.stack((a, b), -1).reshape(28, -1),
                        np.stack((ea, eb), -1).reshape(28, -1))
    qt, st = torch.empty(2 * I, M, dtype=torch.uint8, device="cuda"), torch.empty(M // 128, 2 * I, device="cuda")
    dg.dg_transpose_fp8_blocks(qt, st, kept, skept, block_rows=1, m_indices=mi)
    full = np.zeros((128, 2 * I), np.float32)
    full[:28] = v
    want, ws = orc.quantize(np.ascontiguousarray(full.T), 1)
    assert np.array_equal(qt[:, -128:].cpu().numpy(), want) and np.array_equal(st[-1:].cpu().numpy(), ws)
