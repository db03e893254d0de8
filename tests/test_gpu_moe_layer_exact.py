"""The mixture-of-experts layer keeps its hidden values in FP32: inputs whose
sums are exact in FP32, whatever their order, have to give y exactly.

The gate of every unit is 32, whose silu is 32 in FP32 (e^-32 is below half a
step of 1).  up is a sum of a few integers below 2^24, so h = 32 up w (w a power
of two) is exact and has up to 24 significant bits.  Two neighbouring units
differ in one small term, and each row of W2 takes the difference of such a
pair: a multiple of 16 below 256 * 16, which BF16 holds.  Fewer bits of h
anywhere show in full."""
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


E4M3 = np.array([0x00, 0x38, 0x40, 0x44], dtype=np.uint8)  # 0, 1, 2, 3


def encode(w, fmt):
    """w [E][N][K] of integers -3 .. 3 -> codes and scales, exactly."""
    if fmt == "fp8":
        code = E4M3[np.abs(w).astype(np.int8)] | ((w < 0).astype(np.uint8) << 7)
        E, N, K = w.shape
        return code, np.ones((E, K // 128, -(-N // 128)), dtype=np.float32)
    # a scale of 1/2: codes of 0, 2, 4, 6
    E, N, K = w.shape
    code = np.array([0, 4, 6, 7], dtype=np.uint8)[np.abs(w).astype(np.int8)] | ((w < 0).astype(np.uint8) << 3)
    byte = np.zeros((E, N, -(-K // 128) * 4), dtype=np.uint8)
    byte[..., :K // 32] = 126
    sf = np.ascontiguousarray(byte.view("<i4").transpose(0, 2, 1))
    q = code[..., 0::2] | (code[..., 1::2] << 4)
    assert np.array_equal(ref.values(q[0, :4], sf[0, :, :4]), w[0, :4])
    return q, sf


def call(dg, x, w13, w2, ids, weights, fmt):
    (c13, s13), (c2, s2) = encode(w13, fmt), encode(w2, fmt)
    dev = [torch.from_numpy(np.ascontiguousarray(t)).cuda() for t in (c13, c2, s13, s2, ids, weights)]
    T, H = x.shape
    ws = dg.alloc_workspace(dg.dg_moe_layer_workspace_bytes(T, w13.shape[0], ids.shape[1], H, w2.shape[2]))
    y = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device="cuda")
    dg.dg_moe_layer(y, torch.from_numpy(x).to(torch.bfloat16).cuda(), *dev[:4], *dev[4:], workspace=ws)
    assert not ws[:dg.WORKSPACE_COUNTER_BYTES].any()
    return y.double().cpu().numpy()


SHORT = [(1, 2, 1, 128, 128), (3, 3, 2, 256, 384), (4, 1, 1, 128, 640), (8, 4, 2, 256, 256),
         (16, 1, 1, 128, 384), (17, 3, 2, 128, 1152), (40, 2, 2, 256, 640), (64, 8, 2, 128, 896),
         (64, 2, 2, 256, 1408)]
# hidden units in two chunks and in three
CHUNKS = [(64, 8, 8, 128, 7040), (64, 16, 16, 128, 7040)]
# K blocks of gate/up and of down in every remainder by the depths of the LDS
# rings (a stage is two blocks), from below one round to several; each pair of
# tokens and experts gets other kernels
LONG = [(T, E, k, 128 * n, 128 * m) for T, E, k in ((2, 2, 2), (3, 2, 2), (13, 4, 2), (17, 8, 2), (24, 6, 2),
                                                    (64, 2, 2))
        for n, m in ((2, 17), (3, 16), (5, 14), (7, 12), (9, 9), (11, 7), (13, 5), (15, 4))]
LAYERS = SHORT + CHUNKS + LONG


@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
@pytest.mark.parametrize("T,E,k,H,I", LAYERS)
def test_h_is_not_rounded(dg, T, E, k, H, I, fmt):
    if fmt == "mxfp4":
        H, I = H + 32, I - 32
    rng = np.random.default_rng(T * H + I)
    x = np.zeros((T, H))
    x[:, 0] = 32
    x[:, 1:9] = rng.integers(1, 10, (T, 8)) if k <= 2 else 1
    x[:, 9:] = rng.integers(-255, 256, (T, H - 9)) * 2.0 ** (4 * rng.integers(0, 4, H - 9))
    w13 = np.zeros((E, 2 * I, H), dtype=np.int8)
    w13[:, 0::2, 0] = 1
    few = lambda *shape: (rng.integers(1, 4, shape) * rng.choice([-1, 1], shape)).astype(np.int8)
    # three columns of 9 .. H - 1 for each pair of units, one of 1 .. 8 for its first
    wide = (H - 9) // 3
    cols = 9 + wide * np.arange(3) + rng.integers(0, wide, (E, I // 2, 3))
    same = few(E, I // 2, 3)
    for odd in (1, 3):
        np.put_along_axis(w13[:, odd::4], cols, same, -1)
    np.put_along_axis(w13[:, 1::4], rng.integers(1, 9, (E, I // 2, 1)), few(E, I // 2, 1), -1)
    w2 = np.zeros((E, H, I), dtype=np.int8)
    for e in range(E):
        i = 2 * rng.integers(0, I // 2, H)
        i[:min(H, I // 2)] = 2 * rng.permutation(I // 2)[:H]
        sign = rng.choice([-1, 1], H)
        w2[e, np.arange(H), i], w2[e, np.arange(H), i + 1] = sign, -sign
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    weights = rng.choice([0.5, 1.0, 2.0], (T, k)).astype(np.float32)
    want = np.zeros((T, H))
    for e in range(E):
        t, j = np.nonzero(ids == e)
        up = x[t] @ w13[e, 1::2].astype(np.float64).T
        assert not up.size or np.abs(up).max() < 2 ** 24
        np.add.at(want, t, (32 * up * weights[t, j][:, None]) @ w2[e].astype(np.float64).T)
    assert np.array_equal(want, np.round(want / 16) * 16) and np.abs(want).max() < 4096
    assert np.array_equal(call(dg, x, w13, w2, ids, weights, fmt), want)


@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
@pytest.mark.parametrize("T", [2, 16, 40])
def test_infinite_and_largest_h(dg, T, fmt):
    """h that overflows FP32 is infinite and makes y infinite (not NaN) where
    its weight is not 0; NaN stays NaN; the largest h below that stays finite."""
    E, H, I = 1, 128, 128
    x = np.zeros((T, H))
    x[0, 0] = x[0, 1] = 2.0 ** 70             # unit 0: 2^140
    x[1, 2] = x[1, 3] = 2.0 ** 63             # unit 1: 2^126 (e^-2^63 is 0), three times
    w13, w2 = np.zeros((E, 2 * I, H), dtype=np.int8), np.zeros((E, H, I), dtype=np.int8)
    w13[0, 0, 0] = w13[0, 1, 1] = w13[0, 2, 2] = 1
    w13[0, 3, 3] = 3
    n = np.arange(H)
    w2[0, :, 0] = np.where(n % 2, -1, 1)
    w2[0, :, 1] = np.where(n % 3, -1, 1)
    ids, weights = np.zeros((T, 1), dtype=np.int32), np.ones((T, 1), dtype=np.float32)
    y = call(dg, x, w13, w2, ids, weights, fmt)
    assert np.array_equal(y[0], np.where(n % 2, -np.inf, np.inf))
    assert np.array_equal(y[1], np.where(n % 3, -1, 1) * 3 * 2.0 ** 126)
    assert not y[2:].any()
    x[0, 1] = np.nan
    y = call(dg, x, w13, w2, ids, weights, fmt)
    assert np.isnan(y[0]).all() and np.isfinite(y[1:]).all()


@pytest.mark.parametrize("fmt", ["fp8", "mxfp4"])
@pytest.mark.parametrize("T,E", [(2, 2), (4, 2), (13, 4), (17, 8), (24, 6), (64, 2)])
def test_nan_weights(dg, T, E, fmt):
    """A NaN in an expert's W13 (E4M3: a code, MXFP4: a scale byte) makes y NaN
    for the tokens that chose it, one in W2 its column of y for them; nothing
    else changes."""
    k, H, I = 2, 256, 384
    rng = np.random.default_rng(T)
    w13, w2 = rng.integers(-3, 4, (E, 2 * I, H)), rng.integers(-3, 4, (E, H, I))
    (c13, s13), (c2, s2) = encode(w13, fmt), encode(w2, fmt)
    x = torch.from_numpy(rng.integers(-4, 5, (T, H)) / 256).to(torch.bfloat16).cuda()
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    if E > 2:
        ids[0] = (2, 3)
    ws = dg.alloc_workspace(dg.dg_moe_layer_workspace_bytes(T, E, k, H, I))

    def run():
        d = [torch.from_numpy(np.ascontiguousarray(t)).cuda() for t in (c13, c2, s13, s2, ids)]
        y = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
        dg.dg_moe_layer(y, x, *d, torch.ones(T, k, device="cuda"), workspace=ws)
        return y.double().cpu().numpy()
    want = run()
    assert np.isfinite(want).all()
    if fmt == "fp8":
        c13[0, 2 * 100 + 1, 130], c2[1, 77, 300] = 0x7F, 0xFF
    else:
        s13.view(np.uint8).reshape(E, 2, 2 * I, 4)[0, 1, 2 * 100 + 1, 0] = 255
        s2.view(np.uint8).reshape(E, 3, H, 4)[1, 2, 77, 1] = 255
    want[(ids == 1).any(1), 77] = np.nan
    want[(ids == 0).any(1)] = np.nan
    assert np.array_equal(run(), want, equal_nan=True)
