"""Routing, the grouped layout, dispatch, combine and the 8-bit SwiGLU in plain
64-bit numpy, written from their definitions, and the error bounds the GPU tests
use.

Bounds.  u = 2^-24 is FP32's half step.  BF16 rounds by at most 2^-8 of the
value (its eps / 2), E4M3 by 2^-4 of it, below its normal range (2^-6 of the
scale) by 2^-10 of the scale.
 - e^d in FP32: the argument's rounding moves it by |d| u (one more |d| u where it
   is a difference or a product with a rounded constant), the function by a few
   u.
 - A sum of n terms of FP32: n u sum|terms|.
A value that is quantised after an FP32 computation off by at most e is off by at
most e + 2^-4 (|value| + e) + 2^-10 scale, whichever code it took."""
import numpy as np

U = 2.0 ** -24


def scores(l, scoring):
    """l [T][E] float64 (-inf and NaN: no expert) -> float64."""
    l = np.where(np.isnan(l), -np.inf, l)
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        if scoring == "sigmoid":
            return 1.0 / (1.0 + np.exp(-l))
        m = l.max(1, keepdims=True)
        e = np.where(l > -np.inf, np.exp(l - np.where(m > -np.inf, m, 0.0)), 0.0)
        return e / np.maximum(e.sum(1, keepdims=True), 1e-300)


def route(l, k, bias=None, scoring="softmax", groups=1, top_groups=None, group_best=1,
          renormalise=True, scale=1.0):
    """-> ids int64 [T][k], weights float64 [T][k]"""
    l = np.where(np.isnan(l), -np.inf, np.asarray(l, dtype=np.float64))
    T, E = l.shape
    s = scores(l, scoring)
    off = l == -np.inf
    if bias is not None:
        b = np.asarray(bias, dtype=np.float64)
        off = off | ~(b > -np.inf)[None]
        c = s + np.where(b > -np.inf, b, 0.0)
    else:
        c = s
    key = np.where(off, -np.inf, l if bias is None else c)
    if top_groups is not None and top_groups < groups:
        per = E // groups
        for t in range(T):
            value = np.full(groups, -np.inf)
            for g in range(groups):
                live = np.where(~off[t, g * per:(g + 1) * per])[0] + g * per
                if live.size:
                    v = c[t] if group_best == 2 else key[t]
                    value[g] = np.sort(v[live])[::-1][:group_best].sum()
            for g in np.argsort(-value, kind="stable")[top_groups:]:
                key[t, g * per:(g + 1) * per] = -np.inf
    ids = np.argsort(-key, axis=1, kind="stable")[:, :k]
    none = np.take_along_axis(key, ids, 1) == -np.inf
    # weights from the logits relative to the largest chosen one, free of underflow
    lc = np.where(none, -np.inf, np.take_along_axis(l, ids, 1))
    p = np.where(none, 0.0, np.take_along_axis(s, ids, 1))
    if renormalise:
        with np.errstate(divide="ignore", invalid="ignore"):
            ln = lc if scoring == "softmax" else -np.logaddexp(0.0, -lc)
            top = ln.max(1, keepdims=True)
            p = np.where(none, 0.0, np.exp(ln - np.where(top > -np.inf, top, 0.0)))
        p = p / np.maximum(p.sum(1, keepdims=True), 1e-300)
    return np.where(none, -1, ids), p * scale


def route_bound(l, ids, w, k):
    """Of a weight: e^(l - max) in numerator and denominator, their sums (at most
    26 steps over a wave's lanes and 16 values each), sigmoid and division."""
    lc = np.where(ids >= 0, np.take_along_axis(np.nan_to_num(l, nan=0.0, neginf=0.0, posinf=0.0),
                                               np.maximum(ids, 0), 1), 0.0)
    d = np.abs(np.nan_to_num(l, nan=0.0, neginf=0.0, posinf=0.0)).max(1, keepdims=True) + np.abs(lc)
    return np.abs(w) * (3 * d + 64) * U + 2.0 ** -126


def route_gradient(l, ids, g, scoring="softmax", renormalise=True, scale=1.0):
    """-> d sum(w g) / d l float64 [T][E], and sum|terms| of each."""
    l = np.where(np.isnan(l), -np.inf, np.asarray(l, dtype=np.float64))
    T, E = l.shape
    ok = (ids >= 0) & (ids < E)
    at = np.where(ok, ids, 0)
    ok = ok & (np.take_along_axis(l, at, 1) > -np.inf)
    g = np.where(ok, g, 0.0) * scale
    lc = np.where(ok, np.take_along_axis(l, at, 1), -np.inf)
    d, mag = np.zeros((T, E)), np.zeros((T, E))
    if renormalise:
        with np.errstate(divide="ignore", invalid="ignore"):
            ln = lc if scoring == "softmax" else -np.logaddexp(0.0, -lc)
            top = ln.max(1, keepdims=True)
            q = np.where(ok, np.exp(ln - np.where(top > -np.inf, top, 0.0)), 0.0)
        q = q / np.maximum(q.sum(1, keepdims=True), 1e-300)
        slot = q * (g - (g * q).sum(1, keepdims=True))
        size = q * (np.abs(g) + (np.abs(g) * q).sum(1, keepdims=True))
        if scoring == "sigmoid":
            rest = scores(-np.where(ok, lc, 0.0), "sigmoid")
            slot, size = slot * rest, size * rest
    else:
        s = scores(l, scoring)
        p = np.where(ok, np.take_along_axis(s, at, 1), 0.0)
        if scoring == "softmax":
            slot = size = g * p
            size = np.abs(size)
            d -= s * slot.sum(1, keepdims=True)
            mag += s * size.sum(1, keepdims=True)
        else:
            slot = g * p * scores(-np.where(ok, lc, 0.0), "sigmoid")
            size = np.abs(slot)
    for t, j in zip(*np.nonzero(ok)):
        d[t, ids[t, j]] += slot[t, j]
        mag[t, ids[t, j]] += size[t, j]
    return d, mag


def plan(ids, E, M):
    """-> rows [T][k], pairs [M], m_indices [M], offsets [E + 1], counts [E]"""
    T, k = ids.shape
    rows, pairs, m_indices = np.full((T, k), -1), np.full(M, -1), np.full(M, -1)
    offsets, counts, at = [0], [], 0
    for e in range(E):
        mine = np.nonzero(ids.reshape(-1) == e)[0]
        r = at + np.arange(mine.size)
        rows.reshape(-1)[mine] = r
        pairs[r], m_indices[r] = mine, e
        counts.append(mine.size)
        at += -(-mine.size // 128) * 128
        offsets.append(at)
    return rows, pairs, m_indices, np.array(offsets), np.array(counts)


def blocks_used(m_indices):
    """Rows of 128-row blocks with an expert."""
    return np.repeat(m_indices.reshape(-1, 128)[:, 0] >= 0, 128)


def e4m3(codes):
    c = codes.astype(int)
    ex, man = (c >> 3) & 15, c & 7
    mag = np.where(ex == 0, np.ldexp(man / 8.0, -6), np.ldexp(1 + man / 8.0, ex - 7))
    return np.where((c & 0x7F) == 0x7F, np.nan, np.where(c >= 128, -mag, mag))


def values(q, s):
    """codes [R][C], scales [C/128][R] -> the FP32 numbers they stand for, float64"""
    with np.errstate(over="ignore", invalid="ignore"):  # rows that nothing wrote hold anything
        return (e4m3(q) * np.repeat(s.astype(np.float64).T, 128, axis=1)).astype(np.float32).astype(np.float64)


def sigmoid(x):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-x))


def swiglu(gate, up):
    """-> h, its FP32 error: the sigmoid's (|g| + 2) 2 u, three products"""
    h = gate * sigmoid(gate) * up
    return h, np.abs(h) * (2 * np.abs(gate) + 8) * U + 2.0 ** -126


def swiglu_gradient(gate, up, dh):
    """-> d gate, d up, and their FP32 errors"""
    s = sigmoid(gate)
    r = (2 * np.abs(gate) + 8) * U
    a, b = dh * up * s * (1 + gate * (1 - s)), dh * gate * s
    # 1 - s is off by r s + u, times the silu
    size = np.abs(dh * up) * s * (1 + np.abs(gate) * (1 - s + s))
    return a, b, size * 4 * r + 2.0 ** -126, np.abs(b) * 2 * r + 2.0 ** -126


def check_quantised(q, s, want, err):
    """codes and scales of an FP32 result off by at most err from want."""
    R, C = want.shape
    blocks = np.abs(want).reshape(R, C // 128, 128)
    at = blocks.argmax(-1)
    top = np.take_along_axis(blocks, at[..., None], -1)[..., 0]
    # the largest magnitude is off by no more than the largest error of its block
    e = err.reshape(R, C // 128, 128).max(-1)
    scale = s.astype(np.float64).T
    assert np.all(np.abs(scale * 448 - top) <= e + 4 * U * top + 448 * 2.0 ** -149)
    got = e4m3(q) * np.repeat(scale, 128, axis=1)
    bound = err + 2.0 ** -4 * (np.abs(want) + err) * (1 + 4 * U) + 2.0 ** -10 * np.repeat(scale, 128, axis=1)
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], want[bad][:5])
