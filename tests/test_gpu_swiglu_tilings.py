"""The 8-bit SwiGLU with 4, 8 and (the gradient) 16 rows a workgroup: every row, its scales and
the rows to fill are those of calls on few rows (4 rows a workgroup, each compared with
the definition elsewhere), and rows at the tiles' ends are compared with the definition."""
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


def tile_rows(M, I, backward=False):
    """Rows a workgroup takes."""
    def groups(rows):
        return -(-M // rows) * -(-I // 512)
    if backward and groups(16) >= 4096:
        return 16
    return 4 if groups(8) < 600 else 8


# M, I, grouped, rows a workgroup forward and backward
SHAPES = [(8203, 128, False, 8, 8), (1003, 4224, False, 8, 8), (4801, 128, False, 8, 8), (65537, 128, False, 8, 16),
          (131073, 128, False, 8, 16), (21999, 1152, False, 8, 16), (8320, 128, True, 8, 8), (7296, 1152, True, 8, 8),
          (22016, 1152, True, 8, 16), (44032, 1152, True, 8, 16), (3968, 1152, True, 8, 8), (1536, 1152, True, 4, 4)]


def test_every_tiling_is_there():
    assert [(tile_rows(M, I), tile_rows(M, I, True)) for M, I, *_ in SHAPES] == [tuple(s[3:]) for s in SHAPES]
    for grouped in (False, True):
        assert {rows for s in SHAPES if s[2] == grouped for rows in s[3:]} >= {8, 16}


def spoiled(M, C):
    return (torch.full((M, C), 0x7F, dtype=torch.uint8, device="cuda"),
            torch.full((C // 128, M), -3.0, device="cuda"))


def calls(dg, gu, dh, mi):
    """h alone; h and checkpoint; gradient; gradient and h; gradient in place."""
    M, I = dh.shape
    out = [spoiled(M, I), spoiled(M, I), spoiled(M, 2 * I), spoiled(M, 2 * I), spoiled(M, 2 * I), spoiled(M, I)]
    h, h1, kept, d, d1, h2 = out
    dg.dg_swiglu_fp8(*h, gu, m_indices=mi)
    dg.dg_swiglu_fp8(*h1, gu, *kept, m_indices=mi)
    dg.dg_swiglu_fp8_backward(*d, dh, *kept, m_indices=mi)
    dg.dg_swiglu_fp8_backward(*d1, dh, *kept, *h2, m_indices=mi)
    same = (kept[0].clone(), kept[1].clone())
    dg.dg_swiglu_fp8_backward(*same, dh, *same, m_indices=mi)
    return out + [same]


@pytest.mark.parametrize("M,I,grouped,forward,rows", SHAPES)
def test_tiling(dg, M, I, grouped, forward, rows):
    g = torch.Generator(device="cuda").manual_seed(M)
    rng = np.random.default_rng(M)
    gu = (torch.randn(M, 2 * I, device="cuda", generator=g) * 4).to(torch.bfloat16)
    dh = (torch.randn(M, I, device="cuda", generator=g) * 1e-2).to(torch.bfloat16)
    real, mi = np.ones(M, bool), None
    if grouped:
        m = np.full((M // 128, 128), -1)
        n = rng.choice([0, 1, 3, 31, 33, 100, 127, 128], M // 128)
        m[np.arange(128) < n[:, None]] = 7
        m, real = m.reshape(-1), m.reshape(-1) >= 0
        mi = dev(m.astype(np.int32))
        gu[dev(~real)], dh[dev(~real)] = float("nan"), float("nan")
    got = calls(dg, gu, dh, mi)
    part = 896                       # rows of the calls that it is compared with
    while tile_rows(part, I) > 4:
        part -= 128
    for r in range(0, M, part):
        e = min(M, r + part)
        want = calls(dg, gu[r:e], dh[r:e], None if mi is None else mi[r:e])
        for (q, s), (wq, ws) in zip(got, want):
            assert torch.equal(q[r:e], wq) and torch.equal(s[:, r:e].contiguous().view(torch.int32), ws.view(torch.int32))
    h, h1, kept, d, d1, h2, same = got
    for a, b in ((h, h1), (d, d1), (d, same)):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    if grouped:
        used = ref.blocks_used(m)
        for q, s in got:
            fill, rest = dev(used & ~real), dev(~used)
            assert not q[fill].any() and not s[:, fill].any() and (q[rest] == 0x7F).all() and (s[:, rest] == -3).all()
    # rows at the ends of tiles and some others, against the definition
    ends = np.concatenate([np.arange(8), np.arange(M - 40, M), rows * rng.integers(1, M // rows, 60) - rng.integers(0, 2, 60),
                           rng.integers(0, M, 40)])
    at = np.unique(ends[real[ends]])
    x, y = gu[dev(at)].double().cpu().numpy(), dh[dev(at)].double().cpu().numpy()
    take = lambda o: (o[0][dev(at)].cpu().numpy(), np.ascontiguousarray(o[1][:, dev(at)].cpu().numpy()))
    ref.check_quantised(*take(h), *ref.swiglu(x[:, 0::2], x[:, 1::2]))
    ref.check_quantised(*take(kept), x, np.zeros_like(x))
    v = ref.values(*take(kept))
    a, b, ea, eb = ref.swiglu_gradient(v[:, 0::2], v[:, 1::2], y)
    ref.check_quantised(*take(d), np.stack((a, b), -1).reshape(-1, 2 * I), np.stack((ea, eb), -1).reshape(-1, 2 * I))
    ref.check_quantised(*take(h2), *ref.swiglu(v[:, 0::2], v[:, 1::2]))
