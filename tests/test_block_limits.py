"""Sizes past what a launch holds: host checks of the C ABI (fake addresses, nothing is launched; CPU)."""
import ctypes as C
import os

import pytest

from ragged_grouped_gemm_device_amd import moe as M

pytestmark = pytest.mark.skipif(not os.path.exists(M.LIB_PATH), reason="libmoe.so not built")
F = C.c_void_p(0x1000)


def test_columns_of_4_bit_blocks_past_a_launch_are_refused():
    """256 threads for 64 columns: 2^30 columns would be 2^32 threads, of which a launch keeps none."""
    f = lambda cols, mode: M.load().moe_quant_mxfp4(F, 1, 32, cols, mode, F, F, F, F, None)  # noqa: E731
    assert f(1 << 30, 2) == -2 and f((1 << 30) + 8, 2) == -2 and f(1 << 30, 3) == -2 and f((1 << 31) - 8, 2) == -2
