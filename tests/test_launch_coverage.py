"""Every kernel of the MXFP4 operators and of the mixture-of-experts layer is
launched by some shape of the GPU tests.  The shapes are those lists
themselves; which kernel a shape gets is what the library's own host code does
with them, recorded without a GPU (launch_plan.py)."""
import json
import os
import subprocess
import sys

import pytest

import test_gpu_moe_layer
import test_gpu_moe_layer_exact
import test_gpu_mxfp4
import test_gpu_mxfp4_forms

HERE = os.path.dirname(os.path.abspath(__file__))
LIB = os.path.join(os.path.dirname(HERE), "fp8_block_scaled_dg_amd", "lib", "libdg.so")
BIG = 1 << 40  # a workspace large enough for anything


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("rec") / "librecorder.so")
    subprocess.run(["gcc", "-O1", "-shared", "-fPIC", os.path.join(HERE, "csrc", "launch_recorder.c"),
                    "-o", so], check=True)

    def run(calls):
        r = subprocess.run([sys.executable, os.path.join(HERE, "launch_plan.py"), so, LIB],
                           input=json.dumps(calls), capture_output=True, text=True, check=True)
        out = json.loads(r.stdout)
        assert all(status == 0 for status, _ in out["plans"])
        return out["kernels"], [names for _, names in out["plans"]]
    return run


def quantise(rows, cols):
    for dtype in (0, 1):
        for q, qt in (("p", None), (None, "p"), ("p", "p")):
            yield ["dg_quantize_mxfp4", q, q, qt, qt, "p", dtype, rows, cols, cols, None]
        yield ["dg_dequantize_mxfp4", "p", dtype, "p", "p", rows, cols, None]


def product(M, N, K):
    for ws, n in (("w", BIG), (None, 0)):
        yield ["dg_mxfp4_gemm_nt", "p", "p", "p", "p", "p", M, N, K, ws, n, None]


def bf16a(M, N, K):
    for ws, n in (("w", BIG), (None, 0)):
        yield ["dg_mxfp4_gemm_nt_bf16a", "p", "p", "p", "p", M, N, K, ws, n, None]


def layer(T, E, k, H, I):
    for fmt in (0, 1):
        yield ["dg_moe_layer", "p", "p", "p", "p", "p", "p", fmt, "p", "p", "p", 0, T, E, k, H, I, "w",
               BIG, None]


def shapes_of_the_tests():
    for s in test_gpu_mxfp4.SHAPES + test_gpu_mxfp4_forms.MANY_ROWS:
        yield from quantise(*s)
    for s in (test_gpu_mxfp4.PRODUCTS + test_gpu_mxfp4.SPLIT_PRODUCTS +
              test_gpu_mxfp4_forms.PRODUCTS):
        yield from product(*s)
    for s in test_gpu_mxfp4.BF16A + test_gpu_mxfp4_forms.BF16A:
        yield from bf16a(*s)
    for s in test_gpu_moe_layer.CASES + test_gpu_moe_layer_exact.LAYERS:
        yield from layer(*s)


def test_every_kernel_is_run_by_a_test(plan):
    kernels, plans = plan(list(shapes_of_the_tests()))
    ours = {k for k in kernels if "mxfp4" in k or "moe_" in k}
    assert len(ours) > 30
    missing = ours - {name for names in plans for name in names}
    assert not missing, sorted(missing)


def test_plans_are_the_library_s(plan):
    """The recorder sees real launches: one per product, three per layer, none
    for a refused call."""
    kernels, plans = plan([*product(100, 200, 256), *layer(1, 8, 2, 256, 128)])
    assert [len(p) for p in plans] == [1, 1, 3, 3] and set(sum(plans, [])) <= set(kernels)
