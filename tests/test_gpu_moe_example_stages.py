"""The stages of the example that test_gpu_moe_path.py takes as inputs only: the weights
that routing gives, and the activation between the products."""
import numpy as np
import pytest
import torch

import moe_ref as ref
from gpu_util import need_gpu
from test_gpu_moe_path import dg, example, f64  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,E,k", [(70, 5, 2), (1, 8, 3), (300, 2, 1)])
def test_weights_and_activation(dg, example, T, E, k):  # noqa: F811
    args = ["--tokens", str(T), "--hidden", "384", "--inner", "256", "--experts", str(E), "--k", str(k)]
    layer, x, logits, bias, y, s, dy, g = example.main(args)
    l = f64(logits)
    ids, w = ref.route(l, k, bias=f64(bias), scoring="sigmoid", scale=2.0)
    assert np.array_equal(s["ids"].cpu().numpy(), ids)
    assert np.all(np.abs(f64(s["weights"]) - w) <= ref.route_bound(l, ids, w, k))
    mi = s["plan"].m_indices
    real = mi.cpu().numpy() >= 0
    gu = example.grouped(s["a"], s["sa"], *layer.w13[:2], mi)  # deterministic: the rows that forward had
    rows = f64(gu)[real]
    ref.check_quantised(s["h"].cpu().numpy()[real], np.ascontiguousarray(s["sh"].cpu().numpy()[:, real]),
                        *ref.swiglu(rows[:, 0::2], rows[:, 1::2]))
    ref.check_quantised(s["kept"].cpu().numpy()[real], np.ascontiguousarray(s["skept"].cpu().numpy()[:, real]),
                        rows, np.zeros_like(rows))
