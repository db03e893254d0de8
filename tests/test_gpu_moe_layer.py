"""The mixture-of-experts layer for a few tokens against plain 64-bit numpy
(mxfp4_ref.py, where the bounds are derived)."""
import numpy as np
import pytest
import torch

import mxfp4_ref as ref
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dg():
    need_gpu()
    import fp8_block_scaled_dg_amd as m
    return m


def f64(t):
    return t.double().cpu().numpy()


def fp8_weights(rng, N, K):
    s = rng.uniform(0.5, 2, (K // 128, -(-N // 128))).astype(np.float32) * 2.0 ** -10
    codes = rng.integers(0, 256, (N, K)).astype(np.uint8)
    codes[(codes & 0x7F) > 0x77] = 0x30    # at most 240: keeps NaN out
    return codes, s


def layer(T, E, H, I, fmt, seed):
    rng = np.random.default_rng(seed)
    parts = []
    for n, k in ((2 * I, H), (H, I)):
        one = [(fp8_weights(rng, n, k) if fmt == "fp8" else ref.quantize(rng.standard_normal((n, k)) * 0.05))
               for _ in range(E)]
        parts.append((np.stack([o[0] for o in one]), np.stack([o[1] for o in one])))
    vals = [np.stack([(ref.fp8_values if fmt == "fp8" else ref.values)(c, s) for c, s in zip(*p)])
            for p in parts]
    x = torch.from_numpy(rng.standard_normal((T, H))).to(torch.bfloat16).cuda()
    dev = [torch.from_numpy(np.ascontiguousarray(t)).cuda() for p in parts for t in p]
    return rng, x, dev, vals


def run(dg, x, dev, ids, weights, ws=None, **kw):
    w13, s13, w2, s2 = dev
    T, H = x.shape
    if ws is None:
        ws = dg.alloc_workspace(dg.dg_moe_layer_workspace_bytes(T, w13.shape[0], ids.shape[1], H,
                                                                w13.shape[1] // 2))
    y = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device="cuda")
    dg.dg_moe_layer(y, x, w13, w2, s13, s2, ids, weights, workspace=ws, **kw)
    assert not ws[:dg.WORKSPACE_COUNTER_BYTES].any()
    return y


def empty(T, k):
    return (torch.full((T, k), -7, dtype=torch.int32, device="cuda"),
            torch.full((T, k), float("nan"), device="cuda"))


def check_weights(got, want):
    # exp / sigmoid and the division in FP32: a few ulp of the value, and the
    # rounding of v - max (|v| < 2^5 here) magnified by exp: 2^5 2^-24 each
    assert np.all(np.abs(got - want) <= 2.0 ** -17 * want)


CASES = [(1, 4, 1, 128, 128), (1, 8, 2, 256, 384), (2, 3, 3, 128, 256), (5, 60, 4, 256, 128),
         (13, 16, 8, 384, 256), (16, 2, 1, 128, 128), (40, 2, 2, 256, 128), (64, 1, 1, 128, 256),
         (64, 4, 2, 512, 640), (64, 300, 6, 128, 128), (33, 1000, 16, 128, 128)]


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
@pytest.mark.parametrize("T,E,k,H,I", CASES)
def test_layer(dg, T, E, k, H, I, fmt, scoring):
    if fmt == "mxfp4":
        H, I = H + 32, I - 32
    rng, x, dev, vals = layer(T, E, H, I, fmt, seed=T + E)
    logits = (rng.standard_normal((T, E)) * 2).astype(np.float32)
    ids, weights = empty(T, k)
    y = run(dg, x, dev, ids, weights, logits=torch.from_numpy(logits).cuda(), scoring=scoring)
    want_ids, want_w = ref.route(logits, k, scoring)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    check_weights(f64(weights), want_w)
    ref.check(f64(y), *ref.moe(f64(x), *vals, want_ids, f64(weights)))


@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
def test_masks_ties_and_bad_logits(dg, fmt):
    T, E, k, H, I = 9, 70, 4, 128, 128
    rng, x, dev, vals = layer(T, E, H, I, fmt, seed=5)
    logits = rng.integers(-3, 3, (T, E)).astype(np.float32)     # ties everywhere
    logits[0] = -np.inf                                         # nothing to choose
    logits[1, 2:] = -np.inf                                     # two of four slots
    logits[2, 5:60] = np.nan
    logits[3] = np.finfo(np.float32).min                        # the lowest finite value
    logits[4] = 0.0
    logits[5] = -200.0 - np.arange(E)                           # sigmoids below FP32's range
    logits[6] = 200.0
    logits[7] = np.where(np.arange(E) % 2, -0.0, 0.0)
    for scoring in ("softmax", "sigmoid"):
        ids, weights = empty(T, k)
        y = run(dg, x, dev, ids, weights, logits=torch.from_numpy(logits).cuda(), scoring=scoring)
        want_ids, want_w = ref.route(logits, k, scoring)
        assert np.array_equal(ids.cpu().numpy(), want_ids)
        got = f64(weights)
        assert np.all(np.abs(got - want_w) <= 2.0 ** -14 * want_w + 2.0 ** -126)
        ref.check(f64(y), *ref.moe(f64(x), *vals, want_ids, got))
        assert not f64(y)[0].any()


@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
def test_given_routing(dg, fmt):
    """ids and weights as inputs: empty slots (any id outside the experts),
    one expert twice in a token, everything on one expert (more pairs than
    the row tiles hold), weights zero and negative; inputs stay as they were."""
    T, E, k, H, I = 64, 6, 3, 128, 160 if fmt == "mxfp4" else 128
    rng, x, dev, vals = layer(T, E, H, I, fmt, seed=6)
    for kind in ("mixed", "one", "none"):
        ids = rng.integers(-2, E + 2, (T, k)).astype(np.int32)
        if kind == "one":
            ids[:] = 4
        elif kind == "none":
            ids[:] = np.where(rng.random((T, k)) < 0.5, -1, 2 ** 31 - 1)
        w = rng.standard_normal((T, k)).astype(np.float32)
        w[::5] = 0.0
        di, dw = torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda()
        y = run(dg, x, dev, di, dw)
        ref.check(f64(y), *ref.moe(f64(x), *vals, ids, w.astype(np.float64)), what=kind)
        assert np.array_equal(di.cpu().numpy(), ids) and np.array_equal(dw.cpu().numpy(), w)


def test_masked_inputs_do_not_spread(dg):
    """A token with infinities and NaN spoils its own output only."""
    T, E, k, H, I = 20, 4, 2, 128, 128
    rng, x, dev, vals = layer(T, E, H, I, "mxfp4", seed=7)
    logits = torch.from_numpy((rng.standard_normal((T, E))).astype(np.float32)).cuda()
    ids, weights = empty(T, k)
    clean = run(dg, x, dev, ids, weights, logits=logits).clone()
    x[3, 5], x[11, 0], x[11, 1] = float("nan"), float("inf"), -float("inf")
    y = run(dg, x, dev, ids, weights, logits=logits)
    keep = [t for t in range(T) if t not in (3, 11)]
    assert torch.equal(y[keep], clean[keep])
    assert torch.isnan(y[3]).all()


@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
def test_graph_stream_and_repeat(dg, fmt):
    T, E, k, H, I = 24, 12, 4, 256, 384
    rng, x, dev, _ = layer(T, E, H, I, fmt, seed=8)
    w13, s13, w2, s2 = dev
    logits = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).cuda()
    ids, weights = empty(T, k)
    ws = dg.alloc_workspace(dg.dg_moe_layer_workspace_bytes(T, E, k, H, I))
    want = run(dg, x, dev, ids, weights, ws=ws, logits=logits).clone()
    y = torch.zeros_like(want)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            dg.dg_moe_layer(y, x, w13, w2, s13, s2, ids, weights, logits=logits, workspace=ws)
    for rep in range(3):
        y.zero_(), ids.zero_(), weights.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
        # other work through the same workspace between the replays
        small = run(dg, x[:3].contiguous(), dev, *empty(3, 2), ws=ws, logits=logits[:3].contiguous())
        torch.cuda.synchronize()
        assert torch.isfinite(small).all()
