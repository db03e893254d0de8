"""Widths of the 8-bit SwiGLU whose launch would have 2^24 workgroups of 256 threads
or more are refused on the host, whatever the number of rows."""
import ctypes

import pytest

P = ctypes.c_void_p(0x10000)


@pytest.mark.parametrize("M,I", [(1, (1 << 32) + 128), (1, 1 << 33), (2, 1 << 33), (1, 1 << 34)])
def test_wide_rows_are_refused(M, I):
    import fp8_block_scaled_dg_amd as dg
    assert dg.lib.dg_swiglu_fp8(P, P, None, None, P, None, M, I, None) == 2
    assert dg.lib.dg_swiglu_fp8_backward(P, P, None, None, P, P, P, None, M, I, None) == 2
