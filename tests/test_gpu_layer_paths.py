"""The dense half beside each of the routed experts' paths: permuted copies, gathered rows, MXFP8, and
each activation (GPU). The parts are held against the oracles elsewhere; here the layer's results equal
bit for bit those of the same calls made one by one, with H restored from its codes by hand."""
import numpy as np
import pytest
import torch

from ragged_grouped_gemm_device_amd import workloads as W

from ._util import bf16_tensor

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    from ragged_grouped_gemm_device_amd import moe
    moe.load()
    return moe


def _tensors(wl, n1, ns1, ns):
    rng = np.random.default_rng(wl.seed)
    new = lambda *s, std=1.0: bf16_tensor(W.f32_to_bf16_bits(rng.standard_normal(s).astype(np.float32) * std))  # noqa: E731
    d, n, E = wl.d, wl.n, wl.E
    return dict(x=new(wl.T, d), dout=new(wl.T, d), w1=new(E, d, n1, std=d**-0.5), w2=new(E, n, d, std=n**-0.5),
                wg=new(d, E, std=d**-0.5), s1=new(d, ns1, std=d**-0.5), s2=new(ns, d, std=ns**-0.5))


def _made(M, wl, t, act, ckpt8, mx, h=None):
    gated = act != M.MOE_ACT_SRELU
    buf = M.Buffers(wl.T, wl.k, wl.E, wl.d, wl.n, mx=mx, gated=gated, ckpt8=ckpt8, h=h)
    if mx:
        buf.quantize_weights(t["w1"], t["w2"])
    return buf, M.Router(wl.T, wl.d, wl.E, wl.k, 1, 0.05, 0.01), M.SharedExpert(wl.T, wl.d, 64, act, ckpt8=ckpt8, x8=ckpt8)


@pytest.mark.parametrize("path, act", [(p, a) for p in ("permuted", "gathered", "mx") for a in ("swiglu", "geglu", "srelu")
                                       if (p, a) != ("mx", "srelu")])   # the MXFP8 path is gated
def test_layer_equals_its_parts(M, path, act):
    code = {"swiglu": 0, "geglu": 1, "srelu": 2}[act]
    mx, gather = path == "mx", path == "gathered"
    wl = W.small("paths", 200, 2, 8, 256, 128, seed=21)
    gated = act != "srelu"
    t = _tensors(wl, wl.n * (2 if gated else 1), 64 * (2 if gated else 1), 64)
    fwd, bwd = dict(act=code, gather=gather, mx=mx), dict(act=code, mx=mx, **({"x": t["x"]} if gather else {}))
    buf, router, shared = _made(M, wl, t, code, True, mx)
    r, s = (router, t["wg"]), (shared, t["s1"], t["s2"])
    M.forward(buf, t["x"], None, t["w1"], t["w2"], router=r, shared=s, **fwd)
    buf.h.fill_(float("nan"))
    M.backward(buf, t["dout"], t["w1"], t["w2"], router=r, shared=s, x_tokens=None if gather else t["x"], **bwd)

    one, router1, shared1 = _made(M, wl, t, code, False, mx)
    _, _, shared1 = _made(M, wl, t, code, True, mx)
    router1.project(t["x"], t["wg"])
    M.forward(one, t["x"], router1.logits, t["w1"], t["w2"], **fwd)
    router1.losses(one.topk_idx)
    routed = one.out.clone()
    shared1.forward(t["x"], t["s1"], t["s2"], one.out)
    q, sc = torch.empty_like(one.h, dtype=torch.uint8), torch.empty(one.h.shape[0], one.h.shape[1] // 32, dtype=torch.uint8, device="cuda")
    M.moe_quant_mxfp8(one.h, M.MOE_QUANT_ROWWISE, q, sc)
    M.moe_dequant_mxfp8(q, sc, one.h)
    M.backward(one, t["dout"], t["w1"], t["w2"], logits=router1.logits, **bwd)
    shared1.backward(None, t["dout"], t["s1"], t["s2"], one.dx)
    router1.backward(t["x"], t["wg"], one.dlogits, one.dx)
    torch.cuda.synchronize()
    end = int(buf.offsets[-1])
    assert torch.equal(buf.h[:end], one.h[:end]) and torch.equal(buf.offsets, one.offsets)
    assert not torch.equal(routed, one.out)
    for name in ("out", "dx", "dw1", "dw2", "ds", "dlogits"):
        a, b = getattr(buf, name), getattr(one, name)
        assert torch.isfinite(a).all() and torch.equal(a, b), name
    for name in ("loss", "counts", "prob", "tokens", "dwg", "dlogits16"):
        assert torch.equal(getattr(router, name), getattr(router1, name)), name
    for name in ("z_q", "z_s", "x_q", "x_s", "dw1", "dw2"):
        assert torch.equal(getattr(shared, name), getattr(shared1, name)), name


def test_two_layers_share_the_scratch_that_their_checkpoints_leave_free(M):
    wl = W.small("scratch", 96, 2, 8, 128, 64, seed=22)
    t = _tensors(wl, 128, 128, 64)
    alone = []
    for x in (t["x"], t["dout"]):
        buf, _, _ = _made(M, wl, t, 0, True, False)
        logits = (x.float() @ t["wg"].float()).contiguous()
        M.forward(buf, x, logits, t["w1"], t["w2"])
        M.backward(buf, t["dout"], t["w1"], t["w2"], logits=logits)
        alone.append(buf)
    h = torch.empty_like(alone[0].h)
    both = [_made(M, wl, t, 0, True, False, h)[0] for _ in range(2)]
    for buf, x in zip(both, (t["x"], t["dout"])):
        M.forward(buf, x, (x.float() @ t["wg"].float()).contiguous(), t["w1"], t["w2"])
    for buf, x in zip(reversed(both), (t["dout"], t["x"])):
        M.backward(buf, t["dout"], t["w1"], t["w2"], logits=(x.float() @ t["wg"].float()).contiguous())
    torch.cuda.synchronize()
    for a, b in zip(alone, both):
        assert b.h is h
        for name in ("out", "dx", "dw1", "dw2", "dlogits"):
            assert torch.equal(getattr(a, name), getattr(b, name)), name
