"""FP32 accuracy of the 8-bit SwiGLU and its gradient.  A code hides an error
below 2^-4 of a value; the scale of a block does not: it is its largest
magnitude over 448, in FP32.  Blocks with one hidden unit that is not zero show
that unit's result.

Bounds, in u = 2^-24 of the value.  e^x to one unit in the last place is off by
at most 2 u, 1 + e and the reciprocal round by u each, so the sigmoid by 4 u (of
its denominator's share; below -87 it is e^g itself).  Two products more, and the
scale's division: 7 u, and u for the terms of second order.  A sigmoid below
2^-126 has steps of 2^-149."""
import numpy as np
import pytest
import torch

import moe_ref as ref
from gpu_util import dev, need_gpu

pytestmark = pytest.mark.gpu
STEP = 2.0 ** -149


@pytest.fixture(scope="module")
def dg():
    need_gpu()
    import fp8_block_scaled_dg_amd as m
    return m


def bf16(x):
    return torch.from_numpy(np.asarray(x, dtype=np.float32)).to(torch.bfloat16).cuda()


def lone_units(n):
    """n gates from -104 to 100 with the places of their hidden units."""
    rng = np.random.default_rng(n)
    gate = np.concatenate([rng.uniform(-104, 100, n // 2), rng.standard_normal(n - n // 2) * 3])
    gate[:6] = -90, -88, -87, -86.5, -103, 89
    return rng, gate, rng.integers(0, 128, n)


def close(scales, want, bound):
    """scales * 448 against |want|, off by at most bound and the scale's own step."""
    got = scales.double().cpu().numpy() * 448
    bad = ~(np.abs(got - np.abs(want)) <= bound + 448 * STEP)
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], want[bad][:5], bound[bad][:5])


def test_forward(dg):
    n = 4096
    rng, gate, at = lone_units(n)
    up = rng.standard_normal(n) * 10.0 ** rng.uniform(-3, 3, n)
    up[gate < -60] *= 1e30                       # the sigmoid's far end made visible
    up[:3] = 1e38, 1e30, 1e36
    gu = torch.zeros(n, 256, dtype=torch.bfloat16, device="cuda")
    r = torch.arange(n, device="cuda")
    gu[r, 2 * dev(at)], gu[r, 2 * dev(at) + 1] = bf16(gate), bf16(up)
    h, sh = dg.swiglu_fp8(gu)
    x = gu.double().cpu().numpy()
    g, u = x[np.arange(n), 2 * at], x[np.arange(n), 2 * at + 1]
    want = g * ref.sigmoid(g) * u
    bound = 8 * ref.U * np.abs(want) + np.abs(g * u) * STEP
    close(sh[0], want, bound)
    code = h.cpu().numpy()[np.arange(n), at]
    some = np.abs(want) > bound + 2.0 ** -100  # what the bound leaves apart from 0
    assert (code[some] == np.where(want < 0, 0xFE, 0x7E)[some]).all()


def test_backward(dg):
    """du with up 0 (the block's largest then), dg with a large up, and h again."""
    n = 4096
    rng, gate, at = lone_units(n)
    for scale in (0.0, 100.0):
        up = scale * (1 + rng.random(n)) * np.maximum(np.abs(gate), 1e-3) * rng.choice([-1, 1], n)
        gu = torch.zeros(n, 256, dtype=torch.bfloat16, device="cuda")
        r = torch.arange(n, device="cuda")
        gu[r, 2 * dev(at)], gu[r, 2 * dev(at) + 1] = bf16(gate), bf16(up)
        _, _, kept, skept = dg.swiglu_fp8(gu, keep=True)
        dh = torch.zeros(n, 128, dtype=torch.bfloat16, device="cuda")
        dh[r, dev(at)] = bf16(rng.standard_normal(n) * np.where(gate < -60, 1e30, 1.0))
        d, sd = torch.empty_like(kept), torch.empty_like(skept)
        h, sh = torch.empty(n, 128, dtype=torch.uint8, device="cuda"), torch.empty(1, n, device="cuda")
        dg.dg_swiglu_fp8_backward(d, sd, dh, kept, skept, h, sh)
        v, y = ref.values(kept.cpu().numpy(), skept.cpu().numpy()), dh.double().cpu().numpy()
        i = np.arange(n)
        g, u, y = v[i, 2 * at], v[i, 2 * at + 1], y[i, at]
        sig, rest = ref.sigmoid(g), ref.sigmoid(-g)
        da, db = y * u * sig * (1 + g * rest), y * g * sig
        # dg: sig and 1 - sig (off by 4 u of sig and a rounding), their product with g, the
        # sum and three products
        ea = np.abs(y * u) * sig * ref.U * (10 * (1 + np.abs(g) * rest) + np.abs(g) * (4 * sig + rest))
        ea = ea + np.abs(y * u) * (1 + np.abs(g)) * STEP
        eb = np.abs(db) * 8 * ref.U + np.abs(y * g) * STEP
        scales = sd[dev(2 * at // 128), r]
        close(scales, np.maximum(np.abs(da), np.abs(db)), np.maximum(ea, eb))
        assert (scale > 0) == (np.mean(np.abs(da) > np.abs(db)) > 0.5)
        want = g * sig * u
        close(sh[0], want, 8 * ref.U * np.abs(want) + np.abs(g * u) * STEP)


def test_no_further_off_than_elementary_operations(dg):
    """Over many values the mean error of the blocks' largest is that of the same
    formula in elementary FP32 operations (the same sample of both; a tenth more is
    allowed, 20 deviations of a mean of 2^16 errors)."""
    g = torch.Generator(device="cuda").manual_seed(3)
    M, I = 4096, 2048
    gu = (torch.randn(M, 2 * I, device="cuda", generator=g) * 2).to(torch.bfloat16)
    _, sh = dg.swiglu_fp8(gu)
    x = gu.float()
    a, b = x[:, 0::2], x[:, 1::2]
    top = lambda h: h.view(M, I // 128, 128).abs().amax(-1).t()
    plain = top(a * (1.0 / (1.0 + torch.exp(-a))) * b)
    plain = (plain / torch.full_like(plain, 448.0)).double()
    a, b = a.double(), b.double()
    want = top(a * torch.sigmoid(a) * b) / 448
    error = lambda s: ((s.double() - want).abs() / want).mean().item()
    assert error(sh) <= 1.1 * error(plain)
