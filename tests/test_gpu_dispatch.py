"""The grouped layout, dispatch into it and combine out of it against plain
64-bit numpy (moe_ref.py); codes and scales bit for bit against the oracle's
quantiser."""
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


def choice(rng, T, E, k, how="any"):
    if how == "one":                     # every pair to the last expert
        return np.full((T, k), E - 1)
    ids = np.argsort(rng.random((T, E)) - 0.3 * (np.arange(E) < 2), axis=1)[:, :k]
    if how == "holes":
        ids = np.where(rng.random((T, k)) < 0.3, rng.choice([-1, E, 2 ** 31 - 1, -2 ** 31], (T, k)), ids)
    if how == "twice":
        ids[:, -1] = ids[:, 0]
    return ids


def layout(dg, ids, E, extra=0):
    T, k = ids.shape
    M = dg.dg_moe_plan_rows(T, E, k) + extra
    i32 = dict(dtype=torch.int32, device="cuda")
    out = [torch.full((T, k), -7, **i32), torch.full((M,), -7, **i32), torch.full((M,), -7, **i32),
           torch.full((E + 1,), -7, dtype=torch.int64, device="cuda"), torch.full((E,), -7, **i32)]
    n = dg.dg_moe_plan_workspace_bytes(T, E, k)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda") if n else None
    dg.dg_moe_plan(*out, dev(ids.astype(np.int32)), workspace=ws)
    return dg.MoePlan(*out)


# T, E, k: one launch up to 8192 pairs, then chunks with their counts in the workspace
PLANS = [(1, 1, 1), (1, 8, 2), (1, 1024, 16), (3, 1000, 3), (64, 8, 2), (127, 3, 1), (128, 1, 1), (129, 2, 2), (300, 60, 4),
         (512, 256, 8), (1365, 7, 3), (4097, 5, 1), (2001, 60, 4), (700, 1023, 7), (9001, 256, 8), (40000, 3, 2)]


@pytest.mark.parametrize("how", ["any", "holes", "twice", "one"])
def test_plan(dg, how):
    for n, (T, E, k) in enumerate(PLANS):
        rng = np.random.default_rng(n)
        ids = choice(rng, T, E, k, how)
        extra = 128 * (n % 3)
        p = layout(dg, ids, E, extra)
        inside = np.where((ids >= 0) & (ids < E), ids, -1)
        for got, want in zip(p, ref.plan(inside, E, p.pairs.numel())):
            assert np.array_equal(got.cpu().numpy(), want)


def test_plan_of_nothing(dg):
    p = layout(dg, np.full((5, 2), -1), 4)
    assert (p.rows == -1).all() and (p.pairs == -1).all() and (p.m_indices == -1).all()
    assert not p.offsets.any() and not p.counts.any()


def spoiled(M, H):
    """Buffers with a pattern that no result has (the NaN codes)."""
    return (torch.full((M, H), 0x7F, dtype=torch.uint8, device="cuda"),
            torch.full((H // 128, M), -3.0, device="cuda"))


def check_rows(orc, a, sa, v, p):
    """a, sa hold v's codes at the rows with pairs, zeros up to the block's end,
    and elsewhere what they held; v float32, one row a pair."""
    pairs, mi = p.pairs.cpu().numpy(), p.m_indices.cpu().numpy()
    a, sa = a.cpu().numpy(), sa.cpu().numpy()
    want, ws = orc.quantize(np.ascontiguousarray(v[pairs[pairs >= 0]]), 1)
    assert np.array_equal(a[pairs >= 0], want) and np.array_equal(sa[:, pairs >= 0], ws)
    used = ref.blocks_used(mi)
    fill = used & (pairs < 0)
    assert not a[fill].any() and not sa[:, fill].any()
    assert (a[~used] == 0x7F).all() and (sa[:, ~used] == -3).all()


# T, E, k, H, ldx - H
DISPATCHES = [(1, 8, 2, 128, 0), (1, 4, 1, 7168, 3), (5, 60, 4, 384, 0), (64, 8, 2, 1152, 8), (130, 3, 2, 2048, 13),
              (77, 300, 16, 640, 1), (301, 16, 8, 4224, 0)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("weighted", [False, True])
def test_dispatch(dg, orc, dtype, weighted):
    for n, (T, E, k, H, pad) in enumerate(DISPATCHES):
        rng = np.random.default_rng(n)
        ids = choice(rng, T, E, k, ("any", "holes", "twice", "one")[n % 4])
        p = layout(dg, ids, E, 128 * (n % 2))
        x = torch.from_numpy((rng.standard_normal((T, H + pad)) * 3).astype(np.float32)).to(dtype).cuda()[:, :H]
        x[0, :128] = 0
        x[-1, -128:] = -0.0
        w = rng.standard_normal((T, k)).astype(np.float32)
        w[0, 0] = 0
        v = np.repeat(x.float().cpu().numpy(), k, axis=0)
        if weighted:
            v = w.reshape(-1, 1) * v                  # float32 products
        a, sa = spoiled(p.pairs.numel(), H)
        dg.dg_moe_dispatch_fp8(a, sa, x, p.rows, p.pairs, weights=dev(w) if weighted else None)
        check_rows(orc, a, sa, v, p)


@pytest.mark.parametrize("weighted", [False, True])
def test_dispatch_through_the_workspace(dg, orc, weighted):
    """Enough scales that they meet in the workspace; the call without one gives
    the same bits."""
    T, E, k, H = 2100, 40, 4, 16512
    rng = np.random.default_rng(3)
    ids = choice(rng, T, E, k, "holes")
    p = layout(dg, ids, E, 256)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.randn(T, H, device="cuda", generator=g).to(torch.bfloat16)
    w = torch.rand(T, k, device="cuda", generator=g) if weighted else None
    n = dg.dg_moe_dispatch_fp8_workspace_bytes(T, k, H, weighted)
    assert n > 0
    outs = []
    for ws, stream in ((None, torch.cuda.current_stream().cuda_stream),  # a stream: no workspace
                       (torch.full((n,), 255, dtype=torch.uint8, device="cuda"), None), (None, None)):
        a, sa = spoiled(p.pairs.numel(), H)
        dg.dg_moe_dispatch_fp8(a, sa, x, p.rows, p.pairs, weights=w, workspace=ws, stream=stream)
        outs.append((a, sa))
    for a, sa in outs[1:]:
        assert torch.equal(a, outs[0][0]) and torch.equal(sa, outs[0][1])
    some = torch.arange(0, p.pairs.numel(), 37, device="cuda")  # the oracle on some rows
    rows = some[p.pairs[some] >= 0]
    pair = p.pairs[rows].long()
    v = x[pair // k].float()
    v = w.reshape(-1)[pair][:, None] * v if weighted else v
    want, ws = orc.quantize(v.cpu().numpy(), 1)
    a, sa = outs[1]
    assert np.array_equal(a[rows].cpu().numpy(), want) and np.array_equal(sa[:, rows].cpu().numpy(), ws)
    fill = torch.from_numpy(ref.blocks_used(p.m_indices.cpu().numpy())).cuda() & (p.pairs < 0)
    assert not a[fill].any() and not sa[:, fill].any()
    # the gradient of combine writes the same rows, with and without the weights' gradient
    c = torch.empty(p.pairs.numel(), H, dtype=torch.bfloat16, device="cuda")
    for dw in (None, torch.empty(T, k, device="cuda")):
        for stream in (None, torch.cuda.current_stream().cuda_stream):
            b, sb = spoiled(p.pairs.numel(), H)
            dg.dg_moe_combine_backward(b, sb, dw, x, c, p.rows, p.pairs, w, stream=stream)
            assert torch.equal(a, b) and torch.equal(sa, sb)


# T, E, k, H
PARKED = [(8300, 3, 1, 16512), (4200, 5, 2, 16512), (1100, 16, 8, 16512), (600, 20, 16, 16512)]


@pytest.mark.parametrize("T,E,k,H", PARKED)
def test_combine_backward_through_the_workspace(dg, T, E, k, H):
    """The same bits as without a workspace, with and without weights."""
    g = torch.Generator(device="cuda").manual_seed(k)
    rng = np.random.default_rng(k)
    p = layout(dg, choice(rng, T, E, k, "holes"), E)
    M = p.pairs.numel()
    dy, c = (torch.randn(n, H, device="cuda", generator=g).to(torch.bfloat16) for n in (T, M))
    stream = torch.cuda.current_stream().cuda_stream  # no workspace from torch
    for w in (torch.rand(T, k, device="cuda", generator=g), None):
        assert dg.dg_moe_dispatch_fp8_workspace_bytes(T, k, H, w is not None) > 0
        outs = []
        for s in (stream, None):
            a, sa = spoiled(M, H)
            dw = torch.full((T, k), float("nan"), device="cuda")
            dg.dg_moe_combine_backward(a, sa, dw, dy, c, p.rows, p.pairs, w, stream=s)
            outs.append((a, sa, dw))
        assert all(torch.equal(x, y) for x, y in zip(*outs))


def test_dispatch_of_tiny_and_huge_values(dg, orc):
    """Blocks down to subnormal scales (a -0 and a -tiny keep their sign) and up
    to the largest finite values."""
    rng = np.random.default_rng(11)
    T, H = 90, 256
    x = rng.standard_normal((T, H)).astype(np.float32)
    e = np.concatenate([np.linspace(-150, 126, T - 1).astype(int), [126]])
    with np.errstate(over="ignore", under="ignore"):
        x = np.clip(x, -1.9, 1.9)
        x = (x.astype(np.float64) * np.ldexp(1.0, e)[:, None]).astype(np.float32)
    x[:, ::7] = -0.0
    x[3, :128] = np.float32(2.0 ** -149) * rng.integers(-3, 4, 128).astype(np.float32)
    x[4, :128] = np.float32(2.0 ** -149) * rng.integers(-600, 600, 128).astype(np.float32)
    p = layout(dg, np.zeros((T, 1), dtype=np.int64), 1)
    a, sa = spoiled(p.pairs.numel(), H)
    dg.dg_moe_dispatch_fp8(a, sa, dev(x), p.rows, p.pairs)
    check_rows(orc, a, sa, x, p)


# T, E, k, H
COMBINES = [(1, 1, 1, 8), (1, 8, 2, 4096), (3, 5, 3, 1000), (64, 8, 2, 520), (65, 60, 4, 2048), (33, 40, 16, 72),
            (200, 9, 6, 7168)]


@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("residual", [None, "other", "in place"])
def test_combine(dg, weighted, residual):
    for n, (T, E, k, H) in enumerate(COMBINES):
        rng = np.random.default_rng(n)
        p = layout(dg, choice(rng, T, E, k, ("any", "holes", "twice")[n % 3]), E)
        M = p.pairs.numel()
        c = torch.full((M, H), float("nan"), dtype=torch.bfloat16, device="cuda")  # rows without a pair
        real = p.pairs >= 0
        c[real] = dev(rng.standard_normal((int(real.sum()), H)).astype(np.float32)).to(torch.bfloat16)
        rows = p.rows.cpu().numpy()
        w = np.where(rows >= 0, rng.standard_normal((T, k)), np.nan).astype(np.float32)
        y = torch.full((T, H), 7.0, dtype=torch.bfloat16, device="cuda")
        r = None if residual is None else y if residual == "in place" else torch.randn_like(y)
        add = 0.0 if r is None else r.double().cpu().numpy()
        dg.dg_moe_combine(y, c, p.rows, weights=dev(w) if weighted else None, residual=r)
        t = np.where(rows[..., None] >= 0, c.double().cpu().numpy()[np.maximum(rows, 0)], 0.0)
        if weighted:
            t = t * np.where(rows >= 0, w, 0.0)[..., None]
        want, size = t.sum(1) + add, np.abs(t).sum(1) + np.abs(add)
        err = size * (k + 2) * ref.U
        assert np.all(np.abs(y.double().cpu().numpy() - want) <= err + 2.0 ** -8 * (np.abs(want) + err))


def test_combine_of_nothing(dg):
    p = layout(dg, np.full((3, 2), -1), 2)
    c = torch.full((p.pairs.numel(), 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    assert not dg.moe_combine(c, p).any()
    r = torch.randn(3, 64, device="cuda").to(torch.bfloat16)
    assert torch.equal(dg.moe_combine(c, p, residual=r), r)


# T, E, k, H, lddy - H
BACKWARDS = [(1, 1, 1, 128, 0), (1, 8, 2, 4096, 1), (65, 60, 4, 2048, 0), (33, 40, 16, 384, 5), (100, 9, 6, 7168, 8)]


def test_combine_backward(dg, orc):
    for n, (T, E, k, H, pad) in enumerate(BACKWARDS):
        rng = np.random.default_rng(n)
        p = layout(dg, choice(rng, T, E, k, ("any", "holes")[n % 2]), E)
        M = p.pairs.numel()
        c = torch.full((M, H), float("nan"), dtype=torch.bfloat16, device="cuda")
        real = p.pairs >= 0
        c[real] = dev(rng.standard_normal((int(real.sum()), H)).astype(np.float32)).to(torch.bfloat16)
        dy = dev((rng.standard_normal((T, H + pad)) * 1e-3).astype(np.float32)).to(torch.bfloat16)[:, :H]
        w = rng.random((T, k)).astype(np.float32)
        rows = p.rows.cpu().numpy()
        for parts in ("both", "rows", "weights"):
            dc, sdc = spoiled(M, H) if parts != "weights" else (None, None)
            dw = torch.full((T, k), float("nan"), device="cuda") if parts != "rows" else None
            dg.dg_moe_combine_backward(dc, sdc, dw, dy, c if parts != "rows" else None, p.rows, p.pairs, dev(w))
            if dc is not None:
                check_rows(orc, dc, sdc, w.reshape(-1, 1) * np.repeat(dy.float().cpu().numpy(), k, axis=0), p)
            if dw is not None:
                t = np.where(rows[..., None] >= 0, c.double().cpu().numpy()[np.maximum(rows, 0)], 0.0) \
                    * dy.double().cpu().numpy()[:, None]
                bound = np.abs(t).sum(-1) * (8 * -(-H // 2048) + 10) * ref.U
                assert np.all(np.abs(dw.double().cpu().numpy() - t.sum(-1)) <= bound)


def test_rows_past_32_bits(dg, orc):
    """Rows whose first byte is past 4 GiB, in a layout given by hand."""
    M, H, T = (1 << 20) + 128, 4224, 2
    pairs = torch.full((M,), -1, dtype=torch.int32, device="cuda")
    rows = torch.tensor([[M - 128, 0], [-1, M - 127]], dtype=torch.int32, device="cuda")
    pairs[M - 128], pairs[0], pairs[M - 127] = 0, 1, 3
    x = torch.randn(T, H, device="cuda").to(torch.bfloat16)
    a = torch.empty(M, H, dtype=torch.uint8, device="cuda")
    sa = torch.empty(H // 128, M, device="cuda")
    want, ws = orc.quantize(x.float().cpu().numpy(), 1)
    a.fill_(0x7F)
    dg.dg_moe_dispatch_fp8(a, sa, x, rows, pairs)
    at = torch.tensor([M - 128, 0, M - 127], device="cuda")
    assert np.array_equal(a[at].cpu().numpy(), want[[0, 0, 1]])
    assert np.array_equal(sa[:, at].cpu().numpy(), ws[:, [0, 0, 1]])
    assert not a[M - 126:].any() and not a[1:128].any() and (a[128:256] == 0x7F).all()
    c = torch.empty(M, H, dtype=torch.bfloat16, device="cuda")
    c[at] = torch.randn(3, H, device="cuda").to(torch.bfloat16)
    y = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    dg.dg_moe_combine(y, c, rows)
    assert torch.equal(y, torch.stack((c[M - 128].float() + c[0].float(), c[M - 127].float())).to(torch.bfloat16))


def test_layout_with_holes(dg, orc):
    """A layout that no plan wrote, with rows to fill between those with pairs."""
    for H in (256, 131072):              # the latter through the workspace
        T, k, M = 64, 16, 2048
        rng = np.random.default_rng(H)
        rows = rng.permutation(M)[:T * k].reshape(T, k)
        rows[0] = np.arange(0, M, 128)   # each block's first row has a pair
        pairs, n = np.full(M, -1), np.arange(T * k).reshape(T, k)
        _, first = np.unique(rows[::-1].reshape(-1), return_index=True)
        keep = np.zeros(T * k, bool)
        keep[first] = True
        rows = np.where(keep.reshape(T, k)[::-1], rows, -1)
        pairs[rows[rows >= 0]] = n[rows >= 0]
        x = dev(rng.standard_normal((T, H)).astype(np.float32))
        a, sa = spoiled(M, H)
        assert (dg.dg_moe_dispatch_fp8_workspace_bytes(T, k, H) > 0) == (H > 256)
        dg.dg_moe_dispatch_fp8(a, sa, x, dev(rows.astype(np.int32)), dev(pairs.astype(np.int32)))
        at = np.concatenate([np.nonzero(pairs >= 0)[0][:200], np.nonzero(pairs < 0)[0][:200]])
        q, s = orc.quantize(x.cpu().numpy(), 1)
        want = np.where((pairs[at] >= 0)[:, None], q[pairs[at] // k], 0)
        assert np.array_equal(a[dev(at)].cpu().numpy(), want)
        assert np.array_equal(sa[:, dev(at)].cpu().numpy(), np.where(pairs[at] >= 0, s[:, pairs[at] // k], 0))


def test_foreign_rows_are_left_out(dg):
    """Rows outside [0, M) in a layout that no plan wrote."""
    rows = torch.tensor([[0, 128], [-9, 2 ** 31 - 1]], dtype=torch.int32, device="cuda")
    c = torch.ones(128, 128, dtype=torch.bfloat16, device="cuda")
    y = torch.empty(2, 128, dtype=torch.bfloat16, device="cuda")
    dg.dg_moe_combine(y, c, rows)
    assert (y[0] == 1).all() and not y[1].any()
    pairs = torch.full((128,), -1, dtype=torch.int32, device="cuda")
    pairs[0] = 0
    a, sa = spoiled(128, 128)
    dg.dg_moe_dispatch_fp8(a, sa, y, rows, pairs)
    assert (a[0] == 0x7E).all() and not a[1:].any()
