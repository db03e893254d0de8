"""Every kernel of routing, layout, dispatch, combine and the 8-bit SwiGLU is
launched by some shape of the GPU tests: what the library's host code does with
the tests' own lists, recorded without a GPU (launch_plan.py)."""
import pytest

import test_gpu_dispatch
import test_gpu_route
import test_gpu_swiglu_fp8
from test_launch_coverage import BIG, plan  # noqa: F401  (the recorder)

ENTRIES = ("route_", "plan_", "dispatch_", "combine_", "swiglu_", "transpose_blocks_")


def routing():  # the FP32 argument, scale, has a register of its own: left out
    for T, E, k, G, tg, best in test_gpu_route.CASES:
        for dtype in (0, 1):
            for bias in (None, "p"):
                yield ["dg_moe_route", "p", "p", "p", dtype, E, bias, 0, G, tg, best, 1, T, E, k, None]
            yield ["dg_moe_route_backward", "p", E, "p", "p", "p", dtype, E, 0, 1, T, E, k, None]


def layout():
    for T, E, k in test_gpu_dispatch.PLANS:
        n = T * k
        M = 128 * (min(n, E) + (n - min(n, E)) // 128)
        yield ["dg_moe_plan", "p", "p", "p", "p", "p", "p", T, E, k, M, "w", BIG, None]


def rows():
    big = (2100, 40, 4, 16512, 0)     # test_dispatch_through_the_workspace
    for T, E, k, H, pad in test_gpu_dispatch.DISPATCHES + [big]:
        for w in (None, "p"):
            for ws, n in (("w", BIG), (None, 0)):
                yield ["dg_moe_dispatch_fp8", "p", "p", "p", 1, H + pad, "p", "p", w, T, k, 1024, H, ws, n, None]
    for T, E, k, H in test_gpu_dispatch.COMBINES:
        yield ["dg_moe_combine", "p", "p", "p", None, None, T, k, 1024, H, None]
    for T, E, k, H, pad in test_gpu_dispatch.BACKWARDS + [big] + [(*c, 0) for c in test_gpu_dispatch.PARKED]:
        for dc, dw in (("p", "p"), (None, "p"), ("p", None)):
            yield ["dg_moe_combine_backward", dc, dc, dw, "p", H + pad, "p", "p", "p", "p", T, k, 1024, H, "w", BIG, None]


def activation():
    for M, I, grouped in test_gpu_swiglu_fp8.SHAPES:
        for kept in (None, "p"):
            yield ["dg_swiglu_fp8", "p", "p", kept, kept, "p", None, M, I, None]
            yield ["dg_swiglu_fp8_backward", "p", "p", kept, kept, "p", "p", "p", None, M, I, None]
    for br in (1, 128):
        yield ["dg_transpose_fp8_blocks", "far", "p", br, "p", "p", None, 128, 128, None]


def test_every_kernel_is_run_by_a_test(plan):  # noqa: F811
    calls = [[0x10000000 if a == "far" else a for a in c] for g in (routing, layout, rows, activation) for c in g()]
    kernels, plans = plan(calls)
    ours = {k for k in kernels if any(e in k for e in ENTRIES) and "moe_" not in k}
    assert len(ours) > 40
    missing = ours - {name for names in plans for name in names}
    assert not missing, sorted(missing)
