"""Gradient of routing with masked logits, in every kernel of it (16 lanes a token up
to 256 experts, a wave above), against plain 64-bit numpy.

Bound, in u = 2^-24 of the terms: e^d of a difference d, |d| <= 104 where it is not 0,
is off by (|d| + 2) u, once in a numerator and once in a sum; sums of at most 26 steps,
twice; some ten products: 2 * 106 + 52 + 10.  Results below 2^-126 are not held to it."""
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


def masked(rng, E, low):
    """Rows of logits: nothing left, one left, halves at -inf, NaN or the type's lowest,
    all at the lowest, and logits far below the others."""
    l = (rng.standard_normal((24, E)) * 3).astype(np.float32)
    l[0] = -np.inf
    l[1] = np.nan
    l[2, 1:] = -np.inf
    l[3, :-1] = np.nan
    l[4, ::2] = np.nan
    l[5, ::2] = -np.inf
    l[6] = low
    l[7, :E // 2] = low
    l[8, E // 2:] = low
    l[9, 3:] = -np.inf
    l[10, :E // 2] = -100
    l[11] = -100 - np.arange(E) * 0.5
    l[12, 1::2], l[12, ::4] = -np.inf, np.nan
    for t, fill in zip(range(13, 24), [-np.inf, np.nan, low] * 4):
        l[t, rng.random(E) < 0.5] = fill
    return l


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E", [7, 16, 60, 64, 65, 100, 128, 129, 250, 256, 257, 400, 512, 600, 1024])
def test_masked_logits(dg, E, dtype):
    rng = np.random.default_rng(E)
    k = 6
    logits = torch.from_numpy(masked(rng, E, float(torch.finfo(dtype).min))).to(dtype).cuda()
    l = logits.double().cpu().numpy()
    for scoring in ("softmax", "sigmoid"):
        for renormalise in (True, False):
            kw = dict(scoring=scoring, renormalise=renormalise, scale=1.5)
            ids, _ = ref.route(l, k, **kw)
            assert (ids[0] == -1).all() and (ids[2, 1:] == -1).all()
            # once as routing leaves the slots, once with slots of experts that cannot be chosen
            for at in (ids, np.where(ids < 0, rng.integers(0, E, ids.shape), ids)):
                g = rng.standard_normal(at.shape).astype(np.float32)
                g[:, 0] = np.where(at[:, 0] < 0, np.nan, g[:, 0])  # an empty slot's has no part in it
                d = torch.full((24, E + 1), float("nan"), dtype=dtype, device="cuda")
                dg.dg_moe_route_backward(d[:, :E], dev(g), dev(at.astype(np.int32)), logits, **kw)
                want, size = ref.route_gradient(l, at, np.nan_to_num(g).astype(np.float64), **kw)
                bound = size * 274 * ref.U + 2.0 ** -126
                if dtype == torch.bfloat16:
                    bound = bound + 2.0 ** -8 * (np.abs(want) + bound)
                got = d[:, :E].double().cpu().numpy()
                assert np.all(np.abs(got - want) <= bound)
                assert not got[~(l > -np.inf)].any() and d[:, E].isnan().all()
