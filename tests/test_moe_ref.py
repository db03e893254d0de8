"""The plain forms that the GPU tests of routing and the 8-bit SwiGLU compare
with: definitions by hand, gradients against central differences."""
import numpy as np
import pytest

import moe_ref as ref


def test_route_by_hand():
    inf, nan = np.inf, np.nan
    l = np.array([[0.0, 2, 2, -inf], [-inf] * 4, [nan, 1, -200, -300]])
    ids, w = ref.route(l, 2)
    assert ids.tolist() == [[1, 2], [-1, -1], [1, 2]]
    assert w[0].tolist() == [0.5, 0.5] and not w[1].any()
    ids, w = ref.route(l[2:], 2, scoring="sigmoid", scale=3.0, bias=np.array([0, -inf, 0, 5.0]))
    assert ids.tolist() == [[3, 2]] and np.allclose(w / 3, [[np.exp(-100), 1]], rtol=1e-12)


def test_groups_by_hand():
    # largest single value in group 0, largest pair in group 1
    l = np.log(np.array([[0.4, 0.01, 0.3, 0.29]]))
    assert ref.route(l, 2, groups=2, top_groups=1)[0].tolist() == [[0, 1]]
    assert ref.route(l, 2, groups=2, top_groups=1, group_best=2)[0].tolist() == [[2, 3]]
    # a group with one live expert counts that one; ties go to the first group
    l = np.array([[1.0, -np.inf, 1.0, -np.inf]])
    assert ref.route(l, 2, groups=2, top_groups=1, group_best=2)[0].tolist() == [[0, -1]]


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [True, False])
def test_route_gradient_is_the_difference(scoring, renormalise):
    rng = np.random.default_rng(3)
    l = rng.standard_normal((4, 9)) * 2
    l[1, 3] = -np.inf
    g = rng.standard_normal((4, 3))
    kw = dict(scoring=scoring, renormalise=renormalise, scale=1.5)
    ids, _ = ref.route(l, 3, **kw)
    d, _ = ref.route_gradient(l, ids, g, **kw)
    h = 1e-6
    for t in range(4):
        for e in range(9):
            if l[t, e] == -np.inf:
                assert d[t, e] == 0
                continue
            a, b = l.copy(), l.copy()
            a[t, e] += h
            b[t, e] -= h
            (ia, wa), (ib, wb) = ref.route(a, 3, **kw), ref.route(b, 3, **kw)
            assert np.array_equal(ia, ids) and np.array_equal(ib, ids)
            assert abs(((wa - wb) * g).sum() / (2 * h) - d[t, e]) < 1e-8


def test_swiglu_gradient_is_the_difference():
    rng = np.random.default_rng(4)
    g, u, dh = (rng.standard_normal(2000) * 3 for _ in range(3))
    a, b, _, _ = ref.swiglu_gradient(g, u, dh)
    h = 1e-6
    assert np.allclose(a, dh * (ref.swiglu(g + h, u)[0] - ref.swiglu(g - h, u)[0]) / (2 * h), atol=1e-7)
    assert np.allclose(b, dh * (ref.swiglu(g, u + h)[0] - ref.swiglu(g, u - h)[0]) / (2 * h), atol=1e-7)


def test_plan_by_hand():
    ids = np.array([[1, 0], [1, 1], [-1, 2]])
    rows, pairs, mi, off, cnt = ref.plan(ids, 3, 512)
    assert rows.tolist() == [[128, 0], [129, 130], [-1, 256]]
    assert cnt.tolist() == [1, 3, 1] and off.tolist() == [0, 128, 256, 384]
    assert pairs[[0, 128, 129, 130, 256]].tolist() == [1, 0, 2, 3, 5] and (pairs >= 0).sum() == 5
    assert ref.blocks_used(mi).sum() == 384
