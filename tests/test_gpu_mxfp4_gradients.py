"""The gradients of a linear layer whose products are all in MXFP4, against the
layer without quantisation.

Bound.  With q(.) the quantiser (its errors known exactly from the 64-bit form)
|q(a) q(b)^T - a b^T| <= |q(a) - a| |q(b)|^T + |a| |q(b) - b|^T, to which the
product's own error is added (mxfp4_ref.product).  Each operand is quantised
along the axis that its product contracts over, so a wrong axis or operand, or a
transposed result, is far outside for the operands below, whose rows and columns
differ in size."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import mxfp4_ref as ref
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu


def f64(t):
    return t.double().cpu().numpy()


def quantised(x):
    q, sf = ref.quantize(x)
    return ref.values(q, sf)[:, :x.shape[1]]


def check(got, a, b, what):
    """got = a b^T within the bound, and in the root mean square within half as
    much again as independent errors give."""
    qa, qb = quantised(a), quantised(b)
    want, (_, own) = a @ b.T, ref.product(qa, qb)
    bound = np.abs(qa - a) @ np.abs(qb).T + np.abs(a) @ np.abs(qb - b).T + own
    err = np.abs(got - want)
    assert np.all(err <= bound + 2.0 ** -8 * (np.abs(want) + bound)), what
    # independent errors: their squares add
    spread = (qa - a) ** 2 @ (qb ** 2).T + a ** 2 @ ((qb - b) ** 2).T
    assert np.sqrt(np.mean(err ** 2)) <= 1.5 * np.sqrt(np.mean(spread) + np.mean((2.0 ** -8 * want) ** 2)), what


@pytest.mark.parametrize("M,N,K", [(96, 160, 224), (77, 130, 515), (300, 1000, 160), (1, 64, 96), (65, 33, 31)])
def test_against_the_unquantised_layer(M, N, K):
    need_gpu()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "mxfp4_decoder_block.py")
    spec = importlib.util.spec_from_file_location("mxfp4_decoder_block", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    rng = np.random.default_rng(M + N + K)
    vary = lambda r, c: rng.standard_normal((r, c)) * 2.0 ** rng.integers(-3, 4, (r, 1)) * 2.0 ** rng.integers(-3, 4, c)
    x, w, dy = (torch.from_numpy(vary(*s)).to(torch.bfloat16).cuda() for s in ((M, K), (N, K), (M, N)))
    x.requires_grad_(), w.requires_grad_()
    y = example.Projection.apply(x, w)
    y.backward(dy)
    X, W, D = f64(x.detach()), f64(w.detach()), f64(dy)
    check(f64(y.detach()), X, W, "y")
    check(f64(x.grad), D, W.T, "dx")
    check(f64(w.grad), D.T, X.T, "dw")
