"""A logit of +inf makes its token's softmax weights NaN, and so their gradient: it does
not end as zeros.  The sigmoid of +inf is 1 and its gradient 0."""
import pytest
import torch

from gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dg():
    need_gpu()
    import fp8_block_scaled_dg_amd as m
    return m


@pytest.mark.parametrize("E", [8, 60, 100, 250, 400, 1000])
@pytest.mark.parametrize("renormalise", [True, False])
def test_infinite_logit(dg, E, renormalise):
    l = torch.randn(3, E, device="cuda", generator=torch.Generator(device="cuda").manual_seed(E))
    l[1, 5] = float("inf")
    l[1, 2] = float("-inf")
    g = torch.ones(3, 3, device="cuda")
    for scoring in ("softmax", "sigmoid"):
        ids, w = dg.moe_route(l, 3, scoring=scoring, renormalise=renormalise)
        d = torch.empty_like(l)
        dg.dg_moe_route_backward(d, g, ids, l, scoring=scoring, renormalise=renormalise)
        assert ids[1, 0] == 5 and not d[0].isnan().any() and not d[2].isnan().any()
        if scoring == "sigmoid":
            assert not w.isnan().any() and not d.isnan().any() and d[1, 5] == 0
        else:
            assert w[1].isnan().all() and d[1][ids[1].long()].isnan().all()
            rest = torch.ones(E, dtype=torch.bool, device="cuda")
            rest[ids[1].long()] = False
            assert not d[1][rest].any() if renormalise else d[1].isnan().all()
