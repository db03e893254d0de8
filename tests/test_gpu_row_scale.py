"""The reciprocal and the block scale of the kernels that write E4M3 rows, for every
significand: no difference from the host's correctly rounded divisions."""
import ctypes
import os

import numpy as np
import pytest
import torch

from gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def probe():
    need_gpu()
    import fp8_block_scaled_dg_amd as dg
    lib = ctypes.CDLL(os.path.join(os.path.dirname(dg.__file__), "lib", "libdg_probe.so"))
    lib.dgp_row_scale.argtypes = [ctypes.c_void_p] * 5 + [ctypes.c_int64, ctypes.c_void_p]

    def run(x):
        d = torch.from_numpy(x).cuda()
        out = [torch.full_like(d, float("nan")) for _ in range(4)]
        rc = lib.dgp_row_scale(d.data_ptr(), *(o.data_ptr() for o in out), d.numel(),
                                    torch.cuda.current_stream().cuda_stream)
        assert rc == 0
        return [o.cpu().numpy() for o in out]
    return run


def same(a, b):
    assert np.array_equal(a.view(np.uint32), b.view(np.uint32))


def lift(scale):
    with np.errstate(over="ignore"):
        return np.where(scale < 2.0 ** -62, scale * np.float32(2.0 ** 64), scale).astype(np.float32)


# from the smallest to the largest that occur: scales from 2^-62 (lifted below) to 2^119,
# sums 1 + e^-g to 2^126, and some between
@pytest.mark.parametrize("exponent", [-64, -62, -33, -1, 0, 1, 40, 118, 125])
def test_every_significand(probe, exponent):
    x = (np.arange(1 << 23, dtype=np.uint32) + (np.uint32(exponent + 127) << np.uint32(23))).view(np.float32)
    reciprocal, scale, divisor, inverse = probe(x)
    same(reciprocal, np.float32(1) / x)
    same(scale, x / np.float32(448))
    same(divisor, lift(scale))
    same(inverse, np.float32(1) / lift(scale))


def test_scales_from_subnormal_to_the_largest(probe):
    """Every exponent, subnormal magnitudes and 0 too."""
    rng = np.random.default_rng(0)
    u = rng.integers(0, 0x7F800000, 1 << 20, dtype=np.uint32)
    u[:4] = 0, 1, 0x7F7FFFFF, 0x00800000
    x = u.view(np.float32)
    _, scale, divisor, inverse = probe(x)
    same(scale, x / np.float32(448))
    same(divisor, lift(scale))
    with np.errstate(divide="ignore"):
        same(inverse, np.where(scale > 0, np.float32(1) / lift(scale), np.float32(0)))
