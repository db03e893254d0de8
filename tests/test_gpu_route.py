"""Routing and its gradient against plain 64-bit numpy (moe_ref.py, where the
bounds are derived)."""
import numpy as np
import pytest
import torch

import moe_ref as ref
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dg():
    need_gpu()
    import fp8_block_scaled_dg_amd as m
    return m


def logits_of(rng, T, E, dtype, pad=0):
    """Device logits (rows of a wider tensor where pad is not 0) and their values."""
    l = torch.from_numpy((rng.standard_normal((T, E + pad)) * 2).astype(np.float32)).to(dtype).cuda()[:, :E]
    return l, l.double().cpu().numpy()


def run(dg, logits, k, **kw):
    T = logits.shape[0]
    ids = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), float("nan"), device="cuda")
    dg.dg_moe_route(ids, w, logits, **kw)
    return ids, w


def check(ids, w, l, k, **kw):
    want, ww = ref.route(l, k, **kw)
    got = ids.cpu().numpy()
    assert np.array_equal(got, want)
    assert np.all(np.abs(w.double().cpu().numpy() - ww) <= ref.route_bound(l, want, ww, k))
    return want


# T, E, k, groups, top_groups, group_best
CASES = [(1, 1, 1, 1, 1, 1), (1, 256, 8, 8, 4, 2), (3, 2, 2, 2, 1, 1), (5, 8, 2, 1, 1, 1), (7, 60, 4, 4, 2, 2),
         (4, 64, 8, 8, 3, 1), (9, 65, 6, 5, 2, 2), (33, 96, 16, 3, 2, 2), (16, 128, 8, 16, 5, 2), (6, 129, 3, 1, 1, 1),
         (17, 250, 8, 10, 4, 2), (8, 256, 8, 64, 20, 1), (5, 257, 8, 1, 1, 1), (3, 384, 8, 12, 4, 2),
         (10, 513, 16, 27, 9, 2), (6, 100, 4, 1, 1, 1), (5, 300, 4, 10, 3, 1), (4, 700, 9, 1, 1, 1), (6, 384, 8, 24, 6, 2), (9, 512, 8, 16, 4, 2), (5, 480, 8, 3, 1, 1), (4, 1000, 8, 8, 4, 2), (5, 1024, 16, 64, 7, 2), (70, 16, 3, 8, 2, 1)]


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route(dg, dtype, scoring, bias):
    """BF16 logits tie often: the lowest index has to win."""
    for n, (T, E, k, G, tg, best) in enumerate(CASES):
        rng = np.random.default_rng(100 * n + bias)
        logits, l = logits_of(rng, T, E, dtype, pad=n % 3)
        b = (rng.standard_normal(E) * 0.1).astype(np.float32) if bias else None
        kw = dict(scoring=scoring, groups=G, top_groups=tg, group_best=best, renormalise=n % 2 == 0,
                  scale=1.0 + n % 4)
        ids, w = run(dg, logits, k, bias=torch.from_numpy(b).cuda() if bias else None, **kw)
        ids = check(ids, w, l, k, bias=b, **kw)
        g = rng.standard_normal((T, k)).astype(np.float32)
        d = torch.full((T, E + 3), float("nan"), dtype=dtype, device="cuda")
        grad = {m: kw[m] for m in ("scoring", "renormalise", "scale")}
        dg.dg_moe_route_backward(d[:, :E], torch.from_numpy(g).cuda(), torch.from_numpy(ids.astype(np.int32)).cuda(),
                                 logits, **grad)
        want, size = ref.route_gradient(l, ids, g.astype(np.float64), **grad)
        # scores as in route_bound, on every term; BF16 rounds by 2^-8 of the value
        bound = size * (6 * np.abs(l).max() + 200) * ref.U + 2.0 ** -126
        if dtype == torch.bfloat16:
            bound = bound + 2.0 ** -8 * (np.abs(want) + bound)
        assert np.all(np.abs(d[:, :E].double().cpu().numpy() - want) <= bound)
        assert d[:, E:].isnan().all()


def test_ties_and_equal_logits(dg):
    """All equal, equal pairs, ties at the edge of the choice and between groups."""
    for E, G in ((8, 2), (60, 4), (256, 8), (1024, 16)):
        l = np.zeros((6, E), dtype=np.float32)
        l[1, ::3] = 1
        l[2, E // 2:] = 0.5
        l[3] = np.repeat(np.arange(E // 2), 2)
        l[4] = -np.arange(E) // 5
        l[5, 1] = np.float32(1e-30)
        for bias in (None, np.zeros(E, np.float32)):
            for kw in (dict(), dict(groups=G, top_groups=1), dict(groups=G, top_groups=G - 1, group_best=2)):
                for scoring in ("softmax", "sigmoid"):
                    kw["scoring"] = scoring
                    ids, w = run(dg, torch.from_numpy(l).cuda(), 5, **kw,
                                 bias=None if bias is None else torch.from_numpy(bias).cuda())
                    check(ids, w, l.astype(np.float64), 5, bias=bias, **kw)


def test_close_scores_are_told_apart(dg):
    """Neighbouring FP32 values, and choice values that differ by less than an
    FP32 sum of score and bias would show."""
    rng = np.random.default_rng(5)
    E = 256
    l = np.full((64, E), 1.0, dtype=np.float32)
    for t in range(64):
        at = rng.permutation(E)[:40]
        l[t, at] += rng.integers(-8, 9, 40) * np.float32(2.0 ** -23)
    ids, w = run(dg, torch.from_numpy(l).cuda(), 8)
    check(ids, w, l.astype(np.float64), 8)
    bias = (rng.integers(-4, 5, E) * 2.0 ** -24).astype(np.float32)
    for scoring in ("softmax", "sigmoid"):
        for G in (1, 8):
            kw = dict(scoring=scoring, bias=bias, groups=G, top_groups=max(1, G // 2), group_best=2)
            ids, w = run(dg, torch.from_numpy(l).cuda(), 8, **{**kw, "bias": torch.from_numpy(bias).cuda()})
            check(ids, w, l.astype(np.float64), 8, **kw)


def test_a_few_close_scores(dg):
    """Two to eighteen experts that FP32 does not order, at the top, at the end of
    the choice or below it, among others that are far away."""
    rng = np.random.default_rng(15)
    T = 600
    for E, k in ((60, 4), (256, 8), (500, 16)):
        l = rng.standard_normal((T, E)).astype(np.float32)
        for t in range(T):
            order = np.argsort(-l[t])
            n, at = rng.integers(2, 19), rng.integers(0, k + 4)
            some = order[at:at + n]
            step = rng.choice([2.0 ** -24, 2.0 ** -22, 0.0])
            l[t, some] = l[t, order[at]] + (rng.integers(-6, 7, some.size) * step).astype(np.float32)
        few = (rng.integers(-3, 4, E) * 2.0 ** -23).astype(np.float32)
        for bias in (None, few, (rng.standard_normal(E) * 0.1).astype(np.float32)):
            for scoring in ("softmax", "sigmoid"):
                ids, w = run(dg, torch.from_numpy(l).cuda(), k, scoring=scoring,
                             bias=None if bias is None else torch.from_numpy(bias).cuda())
                check(ids, w, l.astype(np.float64), k, bias=bias, scoring=scoring)


def test_masked_experts(dg):
    """-inf, NaN, the type's lowest value and biases that switch experts off;
    tokens and groups that nothing is left of."""
    rng = np.random.default_rng(6)
    low = float(np.finfo(np.float32).min)
    for E, G in ((16, 4), (250, 10), (600, 6)):
        l = (rng.standard_normal((9, E)) * 2).astype(np.float32)
        l[0] = -np.inf
        l[1, 1:] = -np.inf
        l[2, ::2] = np.nan
        l[3] = low
        l[4, :E // 2] = low
        l[5, E // 4:] = low
        l[6, 3:] = -np.inf
        l[7, :E // 2] = -100
        l[8] = -100 - np.arange(E) * 0.5
        b = (rng.standard_normal(E) * 0.1).astype(np.float32)
        b[5], b[6], b[7], b[8] = -np.inf, np.nan, low, -1e30
        for bias in (None, b):
            for kw in (dict(), dict(groups=G, top_groups=2), dict(groups=G, top_groups=2, group_best=2)):
                for scoring in ("softmax", "sigmoid"):
                    for renormalise in (True, False):
                        kw.update(scoring=scoring, renormalise=renormalise)
                        ids, w = run(dg, torch.from_numpy(l).cuda(), 6, **kw,
                                     bias=None if bias is None else torch.from_numpy(bias).cuda())
                        want = check(ids, w, l.astype(np.float64), 6, bias=bias, **kw)
                        assert (want[0] == -1).all()
    g = rng.standard_normal((9, 6)).astype(np.float32)
    for scoring in ("softmax", "sigmoid"):
        for renormalise in (True, False):
            kw = dict(scoring=scoring, renormalise=renormalise)
            d = torch.full((9, E), float("nan"), device="cuda")
            dg.dg_moe_route_backward(d, torch.from_numpy(g).cuda(), torch.from_numpy(want.astype(np.int32)).cuda(),
                                     torch.from_numpy(l).cuda(), **kw)
            ww, size = ref.route_gradient(l, want, g.astype(np.float64), **kw)
            assert np.all(np.abs(d.double().cpu().numpy() - ww) <= size * (6 * 500 + 200) * ref.U + 2.0 ** -126)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_half_of_the_experts_masked(dg, dtype):
    """A random half of each token's logits at -inf, NaN or the type's lowest
    value, in groups of few experts."""
    rng = np.random.default_rng(16)
    for E, k, G, tg in ((36, 5, 9, 5), (72, 5, 3, 2), (160, 16, 16, 8), (96, 4, 4, 3), (500, 8, 5, 2), (120, 6, 20, 6)):
        for fill in (-np.inf, np.nan, float(torch.finfo(dtype).min)):
            l = (rng.standard_normal((60, E)) * 4).astype(np.float32)
            l[rng.random(l.shape) < 0.5] = fill
            logits = torch.from_numpy(l).to(dtype).cuda()
            l = logits.double().cpu().numpy()
            for bias in (None, np.zeros(E, np.float32), (rng.standard_normal(E) * 0.3).astype(np.float32)):
                for scoring in ("softmax", "sigmoid"):
                    for best in (1, 2):
                        kw = dict(scoring=scoring, groups=G, top_groups=tg, group_best=best, renormalise=best == 1)
                        ids, w = run(dg, logits, k, bias=None if bias is None else torch.from_numpy(bias).cuda(), **kw)
                        check(ids, w, l, k, bias=bias, **kw)


def test_infinite_logit(dg):
    """+inf is chosen first; with the softmax its token's weights are NaN."""
    l = torch.zeros(2, 8)
    l[0, 5] = float("inf")
    for bias in (None, torch.zeros(8, device="cuda")):
        ids, w = run(dg, l.cuda(), 2, bias=bias)
        assert ids.tolist() == [[5, 0], [0, 1]] and w[0].isnan().all() and w[1].tolist() == [0.5, 0.5]
        ids, w = run(dg, l.cuda(), 2, bias=bias, scoring="sigmoid", renormalise=False)
        assert ids.tolist() == [[5, 0], [0, 1]] and w[0].tolist() == [1.0, 0.5]


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [64, 256, 512])
def test_many_tokens(dg, E, scoring):
    rng = np.random.default_rng(7)
    logits, l = logits_of(rng, 2001, E, torch.float32)
    b = (rng.standard_normal(E) * 0.1).astype(np.float32)
    kw = dict(scoring=scoring, groups=8, top_groups=4, group_best=2, scale=2.5)
    ids, w = run(dg, logits, 8, bias=torch.from_numpy(b).cuda(), **kw)
    check(ids, w, l, 8, bias=b, **kw)


def test_rows_far_apart(dg):
    """Offsets past 32 bits."""
    ld = (1 << 30) + 5
    base = torch.empty(2 * ld + 8, device="cuda")
    logits = base.as_strided((3, 8), (ld, 1))
    l = np.random.default_rng(8).standard_normal((3, 8)).astype(np.float32)
    logits.copy_(torch.from_numpy(l))
    ids, w = run(dg, logits, 3)
    ids = check(ids, w, l.astype(np.float64), 3)
    g = np.ones((3, 3), dtype=np.float32) * [[1, 2, 3]]
    dg.dg_moe_route_backward(logits, torch.from_numpy(g.astype(np.float32)).cuda(),
                             torch.from_numpy(ids.astype(np.int32)).cuda(), torch.from_numpy(l).cuda())
    want, size = ref.route_gradient(l, ids, g)
    assert np.all(np.abs(logits.double().cpu().numpy() - want) <= size * 300 * ref.U + 2.0 ** -126)


def test_repeated_and_foreign_ids_in_the_gradient(dg):
    """Slots with the same expert add up; ids outside [0, E) give nothing."""
    rng = np.random.default_rng(9)
    l = rng.standard_normal((3, 12)).astype(np.float32)
    ids = np.array([[4, 4, 1], [12, 2, -5], [2 ** 31 - 1, -1, 99]])
    g = rng.standard_normal((3, 3)).astype(np.float32)
    for scoring in ("softmax", "sigmoid"):
        for renormalise in (True, False):
            d = torch.full((3, 12), float("nan"), device="cuda")
            kw = dict(scoring=scoring, renormalise=renormalise, scale=0.5)
            dg.dg_moe_route_backward(d, torch.from_numpy(g).cuda(), torch.from_numpy(ids.astype(np.int32)).cuda(),
                                     torch.from_numpy(l).cuda(), **kw)
            want, size = ref.route_gradient(l, ids, g.astype(np.float64), **kw)
            assert np.all(np.abs(d.double().cpu().numpy() - want) <= size * 300 * ref.U + 2.0 ** -126)
            assert not d[2].any()
