"""The MXFP4 decoder-block example: its training converges, and its serving
path equals the same path on the dequantised weights."""
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


def test_decoder_block():
    need_gpu()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "mxfp4_decoder_block.py")
    spec = importlib.util.spec_from_file_location("mxfp4_decoder_block", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses, block, x, y, ids, weights = example.main(
        ["--tokens", "5", "--hidden", "256", "--inner", "160", "--experts", "6", "--k", "2"])
    assert all(np.isfinite(losses)) and losses[-1] < 0.1 * losses[0]
    # the projection, then the residual in BF16 as the block forms it
    p = torch.empty_like(x)
    example.dg.dg_mxfp4_gemm_nt_bf16a(p, x, block.w, block.sw)
    ref.check(f64(p), *ref.product(f64(x), ref.values(block.w.cpu().numpy(), block.sw.cpu().numpy())))
    mid = x + p
    values = [np.stack([ref.values(q, s) for q, s in zip(c.cpu().numpy(), sc.cpu().numpy())])
              for c, sc in ((block.w13, block.s13), (block.w2, block.s2))]
    want, bound = ref.moe(f64(mid), *values, ids.cpu().numpy(), f64(weights))
    out = torch.empty_like(x)
    ws = example.dg.alloc_workspace(example.dg.dg_moe_layer_workspace_bytes(5, 6, 2, 256, 160))
    example.dg.dg_moe_layer(out, mid, block.w13, block.w2, block.s13, block.s2, ids, weights,
                            workspace=ws)
    ref.check(f64(out), want, bound)
    assert torch.equal(y, mid + out)
