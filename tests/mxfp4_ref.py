"""MXFP4 and the mixture-of-experts layer in plain 64-bit numpy, written from
the formats' definitions, and the error bounds the GPU tests use.

Bounds.  BF16 rounds by at most 2^-8 of the value.  A sum of n products
accumulated in FP32, in any order and with truncation allowed at every step,
is off by at most n 2^-23 sum|terms|.  The MXFP4 codes, their scales and their
widened values are exact, so nothing else enters the products."""
import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
VALUE = np.concatenate([GRID, -GRID])


def quantize(x):
    """x [R][C] float64 -> codes uint8 [R][ceil(C/32)*16], sf int32
    [ceil(C/128)][R]."""
    x = np.asarray(x, dtype=np.float64)
    R, C = x.shape
    nb, words = -(-C // 32), -(-C // 128)
    v = np.zeros((R, nb * 32))
    v[:, :C] = x
    v = v.reshape(R, nb, 32)
    amax = np.abs(v).max(-1)
    bad = ~np.isfinite(amax)
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.where(amax > 0, np.floor(np.log2(np.where(bad, 1.0, amax))) - 2, -127)
    # log2 may round up just below a power of two
    e = np.where((amax > 0) & ~bad & (np.ldexp(1.0, (e + 2).astype(int)) > amax), e - 1, e)
    e = np.maximum(e, -127).astype(int)
    m = np.abs(v) / np.ldexp(1.0, e)[..., None]
    # nearest of the grid, ties to the even code
    mid = (GRID[1:] + GRID[:-1]) / 2
    with np.errstate(invalid="ignore"):
        code = np.zeros(v.shape, dtype=np.int64)
        for i, t in enumerate(mid):
            code += (m >= t) if i % 2 else (m > t)
    code += np.signbit(v) * 8
    code = np.where(bad[..., None], 0, code).reshape(R, nb * 16, 2)
    q = (code[..., 0] | (code[..., 1] << 4)).astype(np.uint8)
    byte = np.zeros((R, 4 * words), dtype=np.uint8)
    byte[:, :nb] = np.where(bad, 255, e + 127)
    sf = np.ascontiguousarray(byte.view("<i4").T)
    return q, sf


def values(q, sf):
    """codes [R][B], sf [words][R] -> float64 [R][2 B]."""
    R, B = q.shape
    code = np.stack((q & 15, q >> 4), -1).reshape(R, 2 * B)
    byte = np.ascontiguousarray(sf.T).view(np.uint8)[:, :2 * B // 32].astype(int)
    s = np.where(byte == 255, np.nan, np.ldexp(1.0, byte - 127))
    return VALUE[code] * np.repeat(s, 32, axis=1)


def fp8_values(codes, s):
    """E4M3 codes [N][K], scales [K/128][ceil(N/128)] -> float64."""
    c = codes.astype(int)
    ex, man = (c >> 3) & 15, c & 7
    mag = np.where(ex == 0, np.ldexp(man / 8.0, -6), np.ldexp(1 + man / 8.0, ex - 7))
    N = codes.shape[0]
    scale = np.repeat(np.repeat(s.astype(np.float64), 128, axis=0), 128, axis=1)[:, :N].T
    return np.where(c >= 128, -mag, mag) * scale


def product(a, b):
    """C and the bound of its error before the BF16 rounding."""
    return a @ b.T, a.shape[1] * 2.0 ** -23 * (np.abs(a) @ np.abs(b).T)


def check(got, ref, bound, what=""):
    """|got - ref| <= 2^-8 |ref| + (1 + 2^-8) bound, NaN where ref is NaN."""
    nan = np.isnan(ref)
    assert np.array_equal(np.isnan(got), nan), what + ": NaN in the wrong places"
    err = np.where(nan, 0, np.abs(got - ref) - 2.0 ** -8 * np.abs(ref) - (1 + 2.0 ** -8) * bound)
    # 2^-134: half a step of BF16's subnormals
    worst = np.unravel_index(np.argmax(err), err.shape)
    assert err[worst] <= 2.0 ** -134, "%s: %r off by %g (want %g, got %g)" % (
        what, worst, err[worst], ref[worst], got[worst])


def route(logits, k, scoring):
    """ids [T][k], weights [T][k] (float64)."""
    l = np.where(np.isnan(logits), -np.inf, logits.astype(np.float64))
    T, E = l.shape
    ids = np.full((T, k), -1, dtype=np.int32)
    w = np.zeros((T, k))
    for t in range(T):
        order = [e for e in np.argsort(-l[t], kind="stable")[:k] if l[t, e] > -np.inf]
        if not order:
            continue
        v = l[t, order]
        if scoring == "softmax":
            s = np.exp(v - v[0])
        else:  # sig(v) / sig(v0) through logs: log sig(v) = -log(1 + e^-v)
            ls = -np.logaddexp(0.0, -v)
            s = np.exp(ls - ls[0])
        ids[t, :len(order)] = order
        w[t, :len(order)] = s / s.sum()
    return ids, w


def moe(x, w13, w2, ids, weights):
    """x [T][H], w13 [E][2I][H], w2 [E][H][I] float64 -> y and its error bound
    before the last rounding: h is held in two BF16 parts (the second one's
    rounding: 2^-8 of 2^-8), whose products are summed as in product() and
    added, and the FP32 SwiGLU (expf, division, products: 2^-20 with
    room) and weight (given as FP32)."""
    T, H = x.shape
    E, _, I = w2.shape
    y, bound = np.zeros((T, H)), np.zeros((T, H))
    for t in range(T):
        for j, e in enumerate(ids[t]):
            if not 0 <= e < E:
                continue
            gu = w13[e] @ x[t]
            db = H * 2.0 ** -23 * (np.abs(w13[e]) @ np.abs(x[t]))
            g, u, dg, du = gu[0::2], gu[1::2], db[0::2], db[1::2]
            sig = 1 / (1 + np.exp(-g))
            h = g * sig * u * weights[t, j]
            # |silu'| <= 1.1
            dh = np.abs(weights[t, j]) * (1.1 * dg * (np.abs(u) + du) + np.abs(g * sig) * du)
            dh = dh + (2.0 ** -16 + 2.0 ** -20) * (np.abs(h) + dh)
            y[t] += w2[e] @ h
            bound[t] += np.abs(w2[e]) @ (dh + (I + 1) * 2.0 ** -23 * (1 + 2.0 ** -7) * (np.abs(h) + dh))
        bound[t] += 2.0 ** -23 * len(ids[t]) * np.abs(y[t])
    return y, bound
