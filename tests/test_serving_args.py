"""Experts served on 4-bit weights: what the binding lays out and refuses (CPU)."""
import os

import pytest
import torch

from ragged_grouped_gemm_device_amd import moe as M

pytestmark = pytest.mark.skipif(not os.path.exists(M.LIB_PATH), reason="libmoe.so not built")


@pytest.mark.parametrize("form, per", [(M.MOE_X_BF16, 0), (M.MOE_X_MXFP8, 1), (M.MOE_X_MXFP4, 2)])
@pytest.mark.parametrize("act", [M.MOE_ACT_SWIGLU, M.MOE_ACT_SRELU])
def test_sized_shares_the_weights_alone(form, per, act):
    a = M.Experts4(8, 2, 16, 64, 96, act, form, device="cpu")
    b = a.sized(5)
    n1 = 192 if act == M.MOE_ACT_SWIGLU else 96
    assert a.w1_q.shape == (16, n1, 32) and a.w1_s.shape == (16, n1, 2) and a.w2_q.shape == (16, 64, 48) and a.w2_s.shape == (16, 64, 3)
    for name in ("w1_q", "w1_s", "w2_q", "w2_s"):
        assert getattr(a, name) is getattr(b, name)
    assert a.ws.data_ptr() != b.ws.data_ptr()
    for e, T in ((a, 8), (b, 5)):
        assert e.T == T
        if not per:
            assert e.x_q is None and e.a_s is None
            continue
        cap = M.moe_capacity_rows(T, 2, 16)
        assert e.x_q.shape == (T, 64 // per) and e.x_s.shape == (T, 2) and e.a_q.shape == (cap, 96 // per) and e.a_s.shape == (cap, 3)
    if per:
        assert a.a_q.data_ptr() != b.a_q.data_ptr() and a.x_q.data_ptr() != b.x_q.data_ptr()
