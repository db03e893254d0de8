"""FP32 accuracy of the softmax's scores in routing and in its gradient, in u =
2^-24 of the value."""
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


@pytest.mark.parametrize("E", [9, 60, 100, 250, 400, 1000])
def test_gradient_of_far_logits(dg, E):
    """One logit at 0, the others from -85 to -30: their scores sum up to less than
    u / 8, so the sum is 1 and no rounding of it has a part in what is left: e^l (2 u),
    its product with the slots' sum, and for a chosen expert the slot's own product
    (e^l twice, 2 u each, and two roundings) and their sum.  6 u of the terms, and what
    of the sums is below: u / 8 each."""
    rng = np.random.default_rng(E)
    T, k = 257, 5
    l = rng.uniform(-85, -30, (T, E)).astype(np.float32)
    l[np.arange(T), rng.integers(0, E, T)] = 0
    ids, _ = ref.route(l, k)
    g = rng.standard_normal((T, k)).astype(np.float32)
    d = torch.full((T, E), float("nan"), device="cuda")
    dg.dg_moe_route_backward(d, dev(g), dev(ids.astype(np.int32)), dev(l), renormalise=False)
    want, size = ref.route_gradient(l, ids, g.astype(np.float64), renormalise=False)
    assert np.all(np.abs(d.double().cpu().numpy() - want) <= 7 * ref.U * size + 2.0 ** -126)


@pytest.mark.parametrize("E", [60, 250, 500])
def test_weights_no_further_off_than_elementary_operations(dg, E):
    """The mean error of weights that are not renormalised is that of the softmax in
    FP32 (a tenth more is allowed, ten deviations of a mean of 2^16 errors and more)."""
    g = torch.Generator(device="cuda").manual_seed(E)
    l = torch.randn(16384, E, device="cuda", generator=g) * 2
    ids, w = dg.moe_route(l, 4, renormalise=False)
    e = torch.exp(l - l.amax(1, keepdim=True))
    plain = (e / e.sum(1, keepdim=True)).gather(1, ids.long()).double()
    want = torch.softmax(l.double(), 1).gather(1, ids.long())
    error = lambda x: ((x.double() - want).abs() / want).mean().item()
    print(E, error(w) / ref.U, error(plain) / ref.U)
    assert error(w) <= 1.1 * error(plain)
