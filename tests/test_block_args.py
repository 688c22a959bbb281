"""Refusals of the entry points around a MoE block: host checks of the C ABI (fake addresses, nothing is
launched) and of the binding (CPU)."""
import ctypes as C
import os

import pytest
import torch

from ragged_grouped_gemm_device_amd import moe as M

pytestmark = pytest.mark.skipif(not os.path.exists(M.LIB_PATH), reason="libmoe.so not built")
BIG = 1 << 40
BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


def _p(addr=0x1000):
    return C.c_void_p(addr)


F, ODD = _p(), _p(0x1008)


def _routing(score=1, groups=4, kept=2, top=2, renorm=1, scale=1.0):
    return C.byref(M.moe_routing(score, groups, kept, top, renorm, scale))


@pytest.mark.parametrize("kw, want", [
    (dict(T=0), -1), (dict(E=0), -1), (dict(k=0), -1), (dict(k=9), -1), (dict(E=1028), -1), (dict(logits=None), -1),
    (dict(how=None), -1), (dict(how=_routing(score=2)), -2), (dict(how=_routing(groups=3)), -1),
    (dict(how=_routing(groups=0)), -1), (dict(how=_routing(kept=5)), -1), (dict(how=_routing(kept=0)), -1),
    (dict(how=_routing(top=3)), -1), (dict(how=_routing(top=0)), -1), (dict(k=5, how=_routing(kept=2)), -1),
    (dict(how=_routing(scale=float("nan"))), -1), (dict(how=_routing(scale=float("inf"))), -1),
    (dict(E=256, k=65, how=_routing(groups=1, kept=1)), -2), (dict(E=256, how=_routing(groups=128)), -2),
    (dict(idx=None), -1), (dict(src=None), -1), (dict(M_cap=100), -3), (dict(M_cap=1 << 31), -3), (dict(n=0), -3),
    (dict(ws=None), -3), (dict(ws=ODD), -3),
])
def test_route_scores_refusals(kw, want):
    a = dict(logits=F, bias=F, how=_routing(), T=8, E=8, k=2, idx=F, src=F, M_cap=1 << 20, ws=F, n=BIG)
    a.update(kw)
    assert M.load().moe_route_scores(a["logits"], a["bias"], a["how"], a["T"], a["E"], a["k"], a["idx"], F, F, F, F, a["src"],
                                     a["M_cap"], None, a["ws"], a["n"], None) == want
    if want == -3 or "idx" in kw or "src" in kw:
        return
    assert M.load().moe_route_scores_bwd(a["logits"], a["bias"], a["how"], F, F, a["T"], a["E"], a["k"], F, None) == want


def test_route_scores_bwd_refusals():
    f = lambda idx=F, ds=F, d=F, T=8: M.load().moe_route_scores_bwd(F, None, _routing(), idx, ds, T, 8, 2, d, None)  # noqa: E731
    assert f(idx=None) == -1 and f(ds=None) == -1 and f(d=None) == -1 and f(T=(1 << 30) + 1) == -2


@pytest.mark.parametrize("kw, want", [
    (dict(src=None), -1), (dict(batch=0), -1), (dict(R=0), -1), (dict(C=-8), -1), (dict(mode=0), -1), (dict(mode=4), -1),
    (dict(qr=None), -1), (dict(sr=None), -1), (dict(mode=2, qc=None), -1), (dict(mode=2, sc=None), -1), (dict(src=ODD), -1),
    (dict(qr=ODD), -1), (dict(mode=2, qc=ODD), -1), (dict(C=40), -2), (dict(C=36, mode=2), -2), (dict(R=40, mode=2), -2),
    (dict(R=1 << 36), -2), (dict(R=1 << 25, mode=2), -2), (dict(batch=65536), -2),
])
def test_quant_refusals(kw, want):
    a = dict(src=F, batch=1, R=64, C=64, mode=1, qr=F, sr=F, qc=F, sc=F)
    a.update(kw)
    assert M.load().moe_quant_mxfp4(a["src"], a["batch"], a["R"], a["C"], a["mode"], a["qr"], a["sr"], a["qc"], a["sc"], None) == want


def test_dequant_refusals():
    f = lambda q=F, s=F, R=4, Cc=64, o=F: M.load().moe_dequant_mxfp4(q, s, R, Cc, o, None)  # noqa: E731
    assert f(q=None) == -1 and f(s=None) == -1 and f(o=None) == -1 and f(R=0) == -1 and f(Cc=0) == -1
    assert f(q=ODD) == -1 and f(o=ODD) == -1 and f(Cc=40) == -2 and f(R=1 << 40) == -2


@pytest.mark.parametrize("kw, want", [
    (dict(x=None), -1), (dict(wq=None), -1), (dict(ws=None), -1), (dict(off=None), -1), (dict(cnt=None), -1), (dict(y=None), -1),
    (dict(T=0), -1), (dict(k=5), -1), (dict(E=2000), -1), (dict(K=0), -1), (dict(N=-8), -1), (dict(x=ODD), -1), (dict(wq=ODD), -1),
    (dict(y=ODD), -1), (dict(fmt=3), -2), (dict(fmt=-1), -2), (dict(fmt=1), -1), (dict(xs=F), -1), (dict(act=6), -2),
    (dict(act=-1), -2), (dict(K=40), -2), (dict(N=60), -2), (dict(act=0, N=72), -2), (dict(K=(1 << 20) + 32), -2),
    (dict(N=(1 << 20) + 8), -2), (dict(M_cap=100), -3), (dict(M_cap=1 << 31), -3),
    (dict(T=1 << 20, K=2048, src=F, M_cap=1 << 30), -2), (dict(T=1 << 28, k=1, N=1 << 20, M_cap=1 << 30), -2),
])
def test_product_refusals(kw, want):
    a = dict(x=F, xs=None, fmt=0, src=None, T=8, k=2, wq=F, ws=F, off=F, cnt=F, E=4, K=64, N=64, M_cap=1 << 20, act=3, y=F)
    a.update(kw)
    n = M.moe_grouped_linear_mxfp4_workspace_bytes(8, 2, 4, 64, 64)
    assert M.load().moe_grouped_linear_mxfp4(a["x"], a["xs"], a["fmt"], a["src"], a["T"], a["k"], a["wq"], a["ws"], a["off"], a["cnt"],
                                             a["E"], a["K"], a["N"], a["M_cap"], a["act"], a["y"], F, max(n, 16), None) == want


def test_norm_refusals():
    lib = M.load()
    f = lambda x=F, r=None, w=F, T=4, d=64, eps=1e-6, t=None, y=F: lib.moe_norm_fwd(x, r, w, T, d, eps, t, y, None, None)  # noqa: E731
    for kw in (dict(x=None), dict(w=None), dict(y=None), dict(T=0), dict(d=0), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")),
               dict(x=ODD), dict(y=ODD), dict(w=ODD), dict(r=F), dict(t=F), dict(r=ODD, t=F)):
        assert f(**kw) == -1, kw
    for kw in (dict(d=60), dict(d=16392), dict(T=(1 << 30) + 1)):
        assert f(**kw) == -2, kw
    b = lambda dy=F, x=F, w=F, rs=F, T=64, d=64, dx=F, dw=F, ws=F, n=BIG: lib.moe_norm_bwd(  # noqa: E731
        dy, x, w, rs, None, T, d, dx, dw, ws, n, None)
    for kw in (dict(dy=None), dict(x=None), dict(w=None), dict(rs=None), dict(dx=None), dict(dw=ODD), dict(T=0)):
        assert b(**kw) == -1, kw
    assert b(d=60) == -2 and b(ws=None) == -3 and b(n=16) == -3 and b(ws=ODD) == -3


def test_post_norm_refusals():
    lib = M.load()

    def f(y=F, ro=None, tw=None, k=0, x=F, w=F, g=None, gc=0, ga=0, sc=1.0, eps=1e-6, T=4, d=64, t=None, o=F):
        return lib.moe_post_norm_fwd(y, ro, tw, k, x, w, g, gc, ga, sc, eps, T, d, t, o, None, None)

    for kw in (dict(y=None), dict(x=None), dict(w=None), dict(o=None), dict(T=0), dict(eps=0.0), dict(sc=float("inf")), dict(tw=F),
               dict(t=F), dict(ro=F), dict(ro=F, k=1025), dict(g=F), dict(gc=1), dict(g=F, gc=32), dict(g=ODD, gc=64), dict(y=ODD),
               dict(o=ODD)):
        assert f(**kw) == -1, kw
    assert f(d=60) == -2 and f(g=F, gc=1, ga=2) == -2 and f(d=16392) == -2

    def b(do=F, y=F, w=F, rs=F, g=None, gc=0, ga=0, sc=1.0, T=64, d=64, dy=F, dg=None, dw=F, ws=F, n=BIG):
        return lib.moe_post_norm_bwd(do, y, w, rs, g, gc, ga, sc, T, d, dy, dg, dw, ws, n, None)

    for kw in (dict(do=None), dict(y=None), dict(w=None), dict(rs=None), dict(dy=None), dict(dg=F), dict(g=F, gc=64, dg=ODD),
               dict(sc=float("nan")), dict(g=F)):
        assert b(**kw) == -1, kw
    assert b(ga=2) == -2 and b(ws=None) == -3 and b(n=16) == -3


def test_workspace_sizes():
    assert M.moe_route_scores_workspace_bytes(0, 1, 1) == 0 and M.moe_route_scores_workspace_bytes(8, 9, 8) == 0
    assert M.moe_route_scores_workspace_bytes(16, 8, 256) > 0
    assert M.moe_norm_workspace_bytes(0, 64) == 0 and M.moe_norm_workspace_bytes(8, 60) == 0
    assert M.moe_norm_workspace_bytes(1024, 64) > 0


# ------------------------------------------------------------------ binding
def z(*s, t=BF, dev="cpu"):
    return torch.zeros(*s, dtype=t, device=dev)


def _calls(dev):
    n = lambda *s, t=BF: z(*s, t=t, dev=dev)  # noqa: E731
    ws, cap = n(1 << 16, t=U8), M.moe_capacity_rows(6, 2, 8)
    route = (n(6, 2, t=I32), n(6, 2, t=F32), n(8, t=I32), n(9, t=I32), n(12, t=I32), n(cap, t=I32), n(1, t=I32), ws)
    return {
        "moe_route_scores": lambda: M.moe_route_scores(n(6, 8, t=F32), 2, *route, M.Routing(bias=n(8, t=F32))),
        "moe_route_scores_bwd": lambda: M.moe_route_scores_bwd(n(6, 8, t=F32), n(6, 2, t=I32), n(6, 2, t=F32), n(6, 8, t=F32), M.Routing()),
        "moe_quant_mxfp4": lambda: M.moe_quant_mxfp4(n(6, 64), M.MOE_QUANT_ROWWISE, n(6, 32, t=U8), n(6, 2, t=U8)),
        "moe_dequant_mxfp4": lambda: M.moe_dequant_mxfp4(n(6, 32, t=U8), n(6, 2, t=U8), n(6, 64)),
        "moe_grouped_linear_mxfp4": lambda: M.moe_grouped_linear_mxfp4(
            n(cap, 64), n(8, 128, 32, t=U8), n(8, 128, 2, t=U8), n(9, t=I32), n(8, t=I32), n(cap, 128), 6, 2, workspace=ws),
        "moe_norm_fwd": lambda: M.moe_norm_fwd(n(6, 64), n(64), n(6, 64), n(6, t=F32)),
        "moe_norm_bwd": lambda: M.moe_norm_bwd(n(6, 64), n(6, 64), n(64), n(6, t=F32), n(6, 64), n(64, t=F32), ws),
        "moe_post_norm_fwd": lambda: M.moe_post_norm_fwd(n(6, 64), n(6, 64), n(64), n(6, 64), n(6, t=F32), gate=n(6, 1)),
        "moe_post_norm_bwd": lambda: M.moe_post_norm_bwd(n(6, 64), n(6, 64), n(64), n(6, t=F32), n(6, 64), n(64, t=F32), ws,
                                                         gate=n(6, 1), dgate=n(6, 1, t=F32)),
    }


@pytest.mark.parametrize("dev", ["cpu", "meta"])
@pytest.mark.parametrize("name", list(_calls("meta")))
def test_operands_off_the_gpu_are_refused(name, dev):
    with pytest.raises(ValueError, match="GPU"):
        _calls(dev)[name]()


def test_binding_refuses_operands_of_another_shape_type_or_layout():
    f, u = (lambda *s: z(*s, t=F32)), (lambda *s: z(*s, t=U8))
    cap = M.moe_capacity_rows(6, 2, 8)
    ok = dict(x=z(cap, 64), w_q=u(8, 128, 32), w_s=u(8, 128, 2), offsets=z(9, t=I32), counts=z(8, t=I32), y=z(cap, 128), T=6, k=2)
    for bad in (dict(x=z(cap, 72)), dict(x=z(6, 64)), dict(x=u(cap, 64)), dict(x=u(cap, 32)), dict(x=u(cap, 48), x_s=u(cap, 2)),
                dict(x=u(cap, 64), x_s=u(cap, 3)), dict(w_s=u(8, 128, 4)), dict(counts=z(9, t=I32)), dict(offsets=z(8, t=I32)),
                dict(y=z(cap, 64)), dict(act=M.MOE_ACT_SWIGLU), dict(src_of=z(cap, t=I32)), dict(src_of=z(6, t=I32), x=z(6, 64)),
                dict(w_q=u(8, 32, 128).transpose(1, 2)), dict(workspace=u(64)[::2])):
        with pytest.raises(ValueError, match="expected|workspace"):
            M.moe_grouped_linear_mxfp4(**{**ok, **bad})
    route = dict(logits=f(6, 8), k=2, topk_idx=z(6, 2, t=I32), topk_w=f(6, 2), counts=z(8, t=I32), offsets=z(9, t=I32),
                 row_of=z(12, t=I32), src_of=z(cap, t=I32), err_word=None, workspace=u(4096), routing=M.Routing())
    for bad in (dict(logits=z(6, 8)), dict(routing=M.Routing(bias=f(7))), dict(routing=M.Routing(bias=z(8))), dict(topk_idx=z(6, 2, t=torch.int64)),
                dict(topk_w=f(6, 3)), dict(offsets=z(8, t=I32)), dict(row_of=z(6, 2, t=I32)), dict(err_word=z(1))):
        with pytest.raises(ValueError, match="expected"):
            M.moe_route_scores(**{**route, **bad})
    with pytest.raises(ValueError):
        M.moe_quant_mxfp4(z(6, 64), M.MOE_QUANT_ROWWISE, u(6, 64), u(6, 2))
    with pytest.raises(ValueError):
        M.moe_quant_mxfp4(z(64, 6).t(), M.MOE_QUANT_ROWWISE, u(6, 32), u(6, 2))
    with pytest.raises(ValueError):
        M.moe_quant_mxfp4(z(64, 40), M.MOE_QUANT_COLWISE, q_col=u(64, 20), s_col=u(40, 2))
    with pytest.raises(ValueError):
        M.moe_dequant_mxfp4(u(6, 32), u(6, 2), z(6, 32))
    with pytest.raises(ValueError):
        M.moe_norm_fwd(z(6, 64), f(64), z(6, 64))
    with pytest.raises(ValueError):
        M.moe_norm_fwd(z(6, 64), z(64), z(6, 64), residual=z(5, 64), total=z(6, 64))
    with pytest.raises(ValueError):
        M.moe_norm_bwd(z(6, 64), z(6, 64), z(64), z(6), z(6, 64))
    for bad in (dict(gate=z(6, 2)), dict(gate=z(6)), dict(gate=f(6, 1)), dict(total=z(6, 32)), dict(row_of=z(13, t=I32)),
                dict(row_of=z(12, t=I32), topk_w=f(6, 3))):
        with pytest.raises(ValueError):
            M.moe_post_norm_fwd(z(6, 64), z(6, 64), z(64), z(6, 64), **bad)
    for bad in (dict(dgate=f(6, 1)), dict(gate=z(6, 1), dgate=z(6, 1)), dict(gate=z(6, 64), dgate=f(6, 64))):
        with pytest.raises(ValueError):
            M.moe_post_norm_bwd(z(6, 64), z(6, 64), z(64), f(6), z(6, 64), **bad)


def test_backward_after_serving_and_without_the_stream_is_refused():
    buf = M.Buffers(8, 2, 8, 64, 64, device="cpu")
    norms = M.BlockNorms(8, 64, device="cpu")
    with pytest.raises(ValueError, match="x_tokens"):
        M.backward(buf, z(8, 64), z(8, 64, 128), z(8, 64, 64), norms=(norms, z(64), z(64), None))
    buf.served = True
    with pytest.raises(ValueError, match="4-bit"):
        M.backward(buf, z(8, 64), z(8, 64, 128), z(8, 64, 64))
