"""The grouped layout of pairs on both sides of the limit of its single launch (8192),
and of so many (above 131072) that the chunks are more than 512 pairs: a wave then
ranks several rounds of 64, and above a million a thread counts in several turns."""
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


# T, E, k
PLANS = [(8191, 5, 1), (8192, 5, 1), (8193, 5, 1), (4096, 300, 2), (2731, 60, 3), (1025, 1024, 8),
         (131072, 4, 1), (131073, 4, 1), (50000, 7, 3), (20011, 300, 8), (40000, 1024, 16), (70000, 256, 2),
         (150001, 12, 8), (300000, 20, 8)]


@pytest.mark.parametrize("how", ["any", "holes", "one"])
@pytest.mark.parametrize("T,E,k", PLANS)
def test_plan(dg, T, E, k, how):
    rng = np.random.default_rng(T + E)
    ids = rng.integers(0, E, (T, k))                # an expert may stand in several slots
    if how == "holes":
        ids = np.where(rng.random((T, k)) < 0.3, rng.choice([-1, E, 2 ** 31 - 1, -2 ** 31], (T, k)), ids)
    elif how == "one":
        ids[:] = E - 1
    M = dg.dg_moe_plan_rows(T, E, k) + 128 * (T % 2)
    i32 = dict(dtype=torch.int32, device="cuda")
    out = [torch.full((T, k), -7, **i32), torch.full((M,), -7, **i32), torch.full((M,), -7, **i32),
           torch.full((E + 1,), -7, dtype=torch.int64, device="cuda"), torch.full((E,), -7, **i32)]
    n = dg.dg_moe_plan_workspace_bytes(T, E, k)
    assert (n > 0) == (T * k > 8192)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda") if n else None
    dg.dg_moe_plan(*out, dev(ids.astype(np.int32)), workspace=ws)
    inside = np.where((ids >= 0) & (ids < E), ids, -1)
    for got, want in zip(out, plain(inside, E, M)):
        assert np.array_equal(got.cpu().numpy(), want)


def plain(ids, E, M):
    """ref.plan by one stable sort."""
    flat = ids.reshape(-1)
    order = np.argsort(np.where(flat < 0, E, flat), kind="stable")
    order = order[:int((flat >= 0).sum())]
    counts = np.bincount(flat[flat >= 0], minlength=E)
    offsets = np.concatenate(([0], np.cumsum(-(-counts // 128) * 128)))
    rows, pairs, m_indices = np.full(flat.size, -1), np.full(M, -1), np.full(M, -1)
    by = flat[order]
    r = offsets[by] + np.arange(order.size) - (np.cumsum(counts) - counts)[by]
    rows[order], pairs[r], m_indices[r] = r, order, by
    return rows.reshape(ids.shape), pairs, m_indices, offsets, counts


def test_the_plain_form():
    rng = np.random.default_rng(0)
    ids = rng.integers(-1, 9, (200, 3))
    for got, want in zip(plain(ids, 9, 2048), ref.plan(ids, 9, 2048)):
        assert np.array_equal(got, want)
