"""Refusals of the dense entry points: host checks of the C ABI (fake addresses, nothing is
launched) and of the binding (CPU)."""
import ctypes as C
import os

import pytest
import torch

from ragged_grouped_gemm_device_amd import moe as M

pytestmark = pytest.mark.skipif(not os.path.exists(M.LIB_PATH), reason="libmoe.so not built")
BIG = 1 << 40


def _p(addr=0x1000):
    return C.c_void_p(addr)


F, ODD = _p(), _p(0x1008)


def _fwd(x=F, w=F, bias=None, res=None, T=8, K=64, N=64, act=3, f32=0, y=F, z=None, zq=None, zs=None, ws=F, n=BIG):
    return M.load().moe_linear_fwd(x, w, bias, res, T, K, N, act, f32, y, z, zq, zs, ws, n, None)


@pytest.mark.parametrize("kw, want", [
    (dict(x=None), -1), (dict(w=None), -1), (dict(y=None), -1), (dict(T=0), -1), (dict(K=0), -1), (dict(N=-8), -1),
    (dict(act=6), -2), (dict(act=-1), -2), (dict(K=60), -2), (dict(N=60), -2), (dict(act=0, N=96), -2),
    (dict(K=(1 << 20) + 8), -2), (dict(T=1 << 30, N=1 << 20), -2), (dict(T=(1 << 30) + 1, K=8, N=8), -2),
    (dict(x=ODD), -1), (dict(w=ODD), -1), (dict(y=ODD), -1), (dict(bias=ODD), -1), (dict(res=ODD), -1),
    (dict(act=4, z=ODD), -1), (dict(act=4, zq=ODD, zs=F), -1), (dict(act=4, zq=F), -1), (dict(act=4, zs=F), -1),
    (dict(act=4, N=40, zq=F, zs=F), -2), (dict(act=3, z=F), -1), (dict(act=3, zq=F, zs=F), -1),
    (dict(K=8192, ws=None, n=0), -3), (dict(K=8192, n=64), -3), (dict(K=8192, ws=ODD), -3),
])
def test_linear_fwd_refusals(kw, want):
    assert _fwd(**kw) == want


@pytest.mark.parametrize("kw, want", [
    (dict(), -1),                                   # nothing to write
    (dict(dz=F, dy=None), -1), (dict(dbias=F, dy=None), -1), (dict(dz=F, T=0), -1), (dict(dz=F, N=44), -2),
    (dict(dz=F, act=7), -2), (dict(dz=F, act=1, N=96), -2),
    (dict(dz=F, z=None), -1),                       # no z in either form
    (dict(dz=F, zq=F, zs=F), -1),                   # both forms
    (dict(dz=F, z=None, zq=F), -1), (dict(dz=F, z=None, zq=F, zs=F, N=40), -2),
    (dict(dz=F, act=3), -1), (dict(a=F, act=3, z=None), -1),   # no activation: neither z nor a
    (dict(dz=ODD), -1), (dict(a=ODD), -1), (dict(dz=F, dy=ODD), -1), (dict(dz=F, z=ODD), -1),
    (dict(dbias=F, T=4096, ws=None, n=0), -3), (dict(dbias=F, T=4096, n=16), -3),
])
def test_act_bwd_refusals(kw, want):
    a = dict(dy=F, z=F, zq=None, zs=None, T=8, N=64, act=4, dz=None, a=None, dbias=None, ws=F, n=BIG)
    a.update(kw)
    assert M.load().moe_act_bwd(a["dy"], a["z"], a["zq"], a["zs"], a["T"], a["N"], a["act"], a["dz"], a["a"],
                                a["dbias"], a["ws"], a["n"], None) == want


def test_gradient_product_refusals():
    lib = M.load()
    assert lib.moe_linear_dgrad(None, F, None, 8, 64, 64, F, F, BIG, None) == -1
    assert lib.moe_linear_dgrad(F, F, None, 8, 64, 64, None, F, BIG, None) == -1
    assert lib.moe_linear_dgrad(F, F, ODD, 8, 64, 64, F, F, BIG, None) == -1
    assert lib.moe_linear_dgrad(F, F, None, 8, 60, 64, F, F, BIG, None) == -2
    assert lib.moe_linear_dgrad(F, F, None, 8, 64, 8192, F, None, 0, None) == -3
    w = lib.moe_linear_wgrad
    assert w(None, None, None, F, 8, 64, 64, 1, 0, F, F, BIG, None) == -1       # no x in either form
    assert w(F, F, F, F, 8, 64, 64, 1, 0, F, F, BIG, None) == -1                # both forms
    assert w(None, F, None, F, 8, 64, 64, 1, 0, F, F, BIG, None) == -1          # codes without scales
    assert w(None, F, F, F, 8, 40, 64, 1, 0, F, F, BIG, None) == -2             # rows not whole blocks
    assert w(F, None, None, F, 8, 64, 64, 0, 1, F, F, BIG, None) == -2          # accumulation is fp32
    assert w(None, F, F, F, 8192, 64, 64, 1, 0, F, F, 64, None) == -3
    assert w(None, F, F, F, 1000, 2880, 5760, 1, 0, F, F, 1000 * 2880, None) == -3
    assert w(F, None, None, F, 8192, 64, 64, 1, 0, F, None, 0, None) == -3
    assert w(F, None, None, ODD, 8, 64, 64, 1, 0, F, F, BIG, None) == -1


def test_dequant_and_balance_refusals():
    lib = M.load()
    assert lib.moe_dequant_mxfp8(F, F, 0, 32, F, None) == -1
    assert lib.moe_dequant_mxfp8(F, None, 4, 32, F, None) == -1
    assert lib.moe_dequant_mxfp8(ODD, F, 4, 32, F, None) == -1
    assert lib.moe_dequant_mxfp8(F, F, 4, 40, F, None) == -2
    f = lambda T=8, E=4, k=2, S=1, lg=F, seq=None, ws=F, n=BIG: lib.moe_balance_loss(  # noqa: E731
        lg, F, None, seq, T, E, k, S, 1.0, 1.0, F, F, F, F, ws, n, None)
    for kw in (dict(T=0), dict(E=0), dict(E=1025), dict(k=0), dict(k=5), dict(S=0, seq=F), dict(S=9, seq=F),
               dict(S=2), dict(lg=None)):
        assert f(**kw) == -1, kw
    assert f(n=16) == -3 and f(ws=None) == -3 and f(ws=ODD) == -3
    assert f(T=(1 << 30) + 1, E=1, k=1) == -2 and f(T=1 << 28, E=1024, S=1 << 28, seq=F) == -2
    b = lambda T=8, E=4, k=2, S=1, seq=None, d=F: lib.moe_balance_loss_bwd(  # noqa: E731
        F, F, F, None, seq, T, E, k, S, 1.0, 1.0, None, 0, d, None, None)
    assert b(T=0) == -1 and b(k=5) == -1 and b(S=2) == -1 and b(S=9, seq=F) == -1 and b(d=None) == -1


def test_workspace_sizes():
    assert M.moe_linear_workspace_bytes(0, 64, 64) == 0
    assert M.moe_linear_workspace_bytes(8, 60, 64) == 0
    assert M.moe_linear_workspace_bytes(1, 8192, 4096, M.MOE_LINEAR_FWD) > 0
    # a large product from an 8-bit input restores a copy of it there
    assert M.moe_linear_workspace_bytes(1000, 2880, 5760, M.MOE_LINEAR_BWD) >= 1000 * 2880 * 2
    assert M.moe_balance_workspace_bytes(8, 4, 9) == 0
    assert M.moe_balance_workspace_bytes(8, 4, 8) > 0


def test_binding_refuses_operands_of_another_shape_type_or_layout():
    bf = torch.bfloat16
    x, w, y = torch.zeros(4, 64, dtype=bf), torch.zeros(64, 128, dtype=bf), torch.zeros(4, 128, dtype=bf)
    with pytest.raises(ValueError):
        M.moe_linear_fwd(x, w, y[:, :64], M.MOE_ACT_NONE)            # y of another width
    with pytest.raises(ValueError):
        M.moe_linear_fwd(x, w, y, M.MOE_ACT_SWIGLU)                  # gated: y [4, 64]
    with pytest.raises(ValueError):
        M.moe_linear_fwd(x, w.t().contiguous(), y)                   # [N, K]
    with pytest.raises(ValueError):
        M.moe_linear_fwd(x, torch.zeros(128, 64, dtype=bf).t(), y)   # not dense
    with pytest.raises(ValueError):
        M.moe_linear_fwd(x.float(), w, y)
    with pytest.raises(ValueError):
        M.moe_linear_fwd(x, w, y, bias=torch.zeros(128))             # bias is bf16
    with pytest.raises(ValueError):
        M.moe_linear_fwd(x, w, y, M.MOE_ACT_GELU, z_q=torch.zeros(4, 128, dtype=torch.uint8),
                         z_s=torch.zeros(4, 3, dtype=torch.uint8))
    with pytest.raises(ValueError):
        M.moe_linear_wgrad(x, y[:3], torch.zeros(64, 128))
    with pytest.raises(ValueError):
        M.moe_linear_dgrad(y, w, torch.zeros(5, 64, dtype=bf))
    with pytest.raises(ValueError):
        M.moe_act_bwd(y, None, M.MOE_ACT_NONE, dbias=torch.zeros(64))
    with pytest.raises(ValueError):
        M.moe_act_bwd(None, y)
    lg, idx = torch.zeros(6, 4), torch.zeros(6, 2, dtype=torch.int32)
    one = dict(loss=torch.zeros(3), counts=torch.zeros(1, 4, dtype=torch.int32), prob=torch.zeros(1, 4),
               tokens=torch.zeros(3, dtype=torch.int32), workspace=torch.zeros(4096, dtype=torch.uint8),
               balance_coef=1.0, z_coef=1.0)
    for bad in (dict(counts=torch.zeros(1, 5, dtype=torch.int32)), dict(tokens=torch.zeros(2, dtype=torch.int32)),
                dict(valid=torch.zeros(5, dtype=torch.uint8)), dict(valid=torch.zeros(6)),
                dict(seq_offsets=torch.zeros(3, dtype=torch.int32)),
                dict(seq_offsets=torch.zeros(2, dtype=torch.int64))):
        with pytest.raises(ValueError):
            M.moe_balance_loss(lg, idx, **{**one, **bad})
    with pytest.raises(ValueError):
        M.moe_balance_loss(lg, idx.long(), **one)


def test_binding_refuses_more_rows_than_the_abi_counts():
    """Row counts past 32 bits would wrap to another, valid one (meta tensors: nothing is allocated)."""
    n, bf = (1 << 32) + 8, torch.bfloat16
    new = lambda *s, t=bf: torch.empty(*s, dtype=t, device="meta")  # noqa: E731
    with pytest.raises(ValueError, match="rows"):
        M.moe_linear_fwd(new(n, 8), new(8, 8), new(n, 8))
    with pytest.raises(ValueError, match="rows"):
        M.moe_act_bwd(new(n, 8), new(n, 8))
    with pytest.raises(ValueError, match="rows"):
        M.moe_linear_dgrad(new(n, 8), new(8, 8), new(n, 8))
    with pytest.raises(ValueError, match="rows"):
        M.moe_linear_wgrad(new(n, 8), new(n, 8), new(8, 8))
    i32, f32 = torch.int32, torch.float32
    with pytest.raises(ValueError, match="rows"):
        M.moe_balance_loss(new(n, 4, t=f32), new(n, 2, t=i32), new(3, t=f32), new(1, 4, t=i32), new(1, 4, t=f32),
                           new(3, t=i32), new(64, t=torch.uint8), 1.0, 1.0)
    with pytest.raises(ValueError, match="rows"):
        M.moe_balance_loss_bwd(new(n, 4, t=f32), new(1, 4, t=i32), new(3, t=i32), new(n, 4, t=f32), 2, 1.0, 1.0)


def test_buffers_refuse_a_scratch_of_another_shape_or_type():
    cap = M.moe_capacity_rows(8, 2, 4)
    ok = torch.empty(cap, 128, dtype=torch.bfloat16)
    assert M.Buffers(8, 2, 4, 64, 64, device="cpu", ckpt8=True, h=ok).h is ok
    for bad in (ok[:-1], ok[:, :64], ok.float(), ok.t().contiguous().t()):
        with pytest.raises(ValueError, match="h:"):
            M.Buffers(8, 2, 4, 64, 64, device="cpu", ckpt8=True, h=bad)
