"""Routing with scores and the block's norms beside each of the routed experts' paths: permuted copies, gathered rows,
MXFP8 and 8-bit checkpoints of H (GPU). The parts are held against the oracles elsewhere; here a block's results equal
bit for bit those of the same calls made one by one."""
import numpy as np
import pytest
import torch

from oracle import block_oracle as B
from ragged_grouped_gemm_device_amd import workloads as W

from ._util import bf16_tensor, f32_tensor

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
EPS, SCALE = 1e-6, 0.5


@pytest.fixture(scope="module")
def M():
    from ragged_grouped_gemm_device_amd import moe
    moe.load()
    return moe


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("path, act", [("permuted", "swiglu"), ("gathered", "srelu"), ("mx", "swiglu"), ("mx", "geglu"), ("ckpt8", "geglu"),
                                       ("mx ckpt8", "swiglu")])
def test_block_equals_its_parts(M, path, act, score):
    code = {"swiglu": 0, "geglu": 1, "srelu": 2}[act]
    mx, gather, ckpt8 = "mx" in path, path == "gathered", "ckpt8" in path
    wl = W.small("block-paths", 200, 2, 8, 256, 128, seed=31)
    T, E, d, k = wl.T, wl.E, wl.d, wl.k
    rng = np.random.default_rng(wl.seed)
    new = lambda *s, std=1.0, mean=0.0: bf16_tensor(W.f32_to_bf16_bits((rng.standard_normal(s) * std + mean).astype(np.float32)))  # noqa: E731
    x, dout, gate, wa, wb = new(T, d), new(T, d), new(T, d), new(d, std=0.2, mean=1.0), new(d, std=0.2, mean=1.0)
    gated = act != "srelu"
    w1, w2, wg = new(E, d, wl.n * (2 if gated else 1), std=d**-0.5), new(E, wl.n, d, std=wl.n**-0.5), new(d, E, std=d**-0.5)
    bias = (rng.standard_normal(E) * 0.05).astype(np.float32)
    routing = M.Routing(M.MOE_SCORE_SIGMOID if score == "sigmoid" else M.MOE_SCORE_SOFTMAX, f32_tensor(bias), 4, 2, 2, True, 1.5)

    def made():
        buf = M.Buffers(T, k, E, d, wl.n, mx=mx, gated=gated, ckpt8=ckpt8)
        if mx:
            buf.quantize_weights(w1, w2)
        # the balance loss is a softmax's; the z loss goes with both
        return buf, M.Router(T, d, E, k, 1, 0.05 if score == "softmax" else 0.0, 0.01)

    buf, router = made()
    norms = M.BlockNorms(T, d, d, M.MOE_GATE_SIGMOID, SCALE, EPS)
    kw = dict(router=(router, wg), routing=routing, norms=(norms, wa, wb, gate), act=code, mx=mx)
    M.forward(buf, x, None, w1, w2, gather=gather, **kw)
    if ckpt8:
        buf.h.fill_(float("nan"))
    M.backward(buf, dout, w1, w2, **kw, **({"x": x} if gather else {"x_tokens": x}))

    one, router1 = made()
    full = lambda *s, t=BF: torch.full(s, float("nan"), dtype=t, device="cuda")  # noqa: E731
    y, out, dy, dx, dgate = (full(T, d) for _ in range(5))
    ra, rb, dwa, dwb = full(T, t=F32), full(T, t=F32), full(d, t=F32), full(d, t=F32)
    ws = torch.empty(max(16, M.moe_norm_workspace_bytes(T, d)), dtype=torch.uint8, device="cuda")
    M.moe_norm_fwd(x, wa, y, ra, EPS)
    router1.project(y, wg)
    M.forward(one, y, router1.logits, w1, w2, routing=routing, act=code, mx=mx, gather=gather)
    router1.losses(one.topk_idx)
    M.moe_post_norm_fwd(one.out, x, wb, out, rb, EPS, gate=gate, gate_act=M.MOE_GATE_SIGMOID, scale=SCALE)
    M.moe_post_norm_bwd(dout, one.out, wb, rb, dy, dwb, ws, gate=gate, dgate=dgate, gate_act=M.MOE_GATE_SIGMOID, scale=SCALE)
    M.backward(one, dy, w1, w2, logits=router1.logits, routing=routing, act=code, mx=mx, **({"x": y} if gather else {}))
    # the routing's own share, by itself
    dlogits = full(T, E, t=F32)
    M.moe_route_scores_bwd(router1.logits, one.topk_idx, one.ds, dlogits, routing)
    assert torch.equal(dlogits, one.dlogits)
    idx, w = B.route_scores(router1.logits.cpu().numpy(), bias, score, k, 4, 2, 2, True, 1.5)
    assert np.array_equal(one.topk_idx.cpu().numpy(), idx)
    np.testing.assert_allclose(one.topk_w.cpu().numpy(), w, rtol=16 * 2.0**-24)
    router1.backward(y, wg, one.dlogits, one.dx)
    M.moe_norm_bwd(one.dx, x, wa, ra, dx, dwa, ws, dres=dout)
    torch.cuda.synchronize()
    for name in ("out", "dx", "dw1", "dw2", "ds", "dlogits", "topk_idx", "topk_w"):
        a, b = getattr(buf, name), getattr(one, name)
        assert torch.isfinite(a).all() and torch.equal(a, b), name
    for name in ("loss", "counts", "prob", "dwg"):
        assert torch.equal(getattr(router, name), getattr(router1, name)), name
    for a, b in ((norms.y, y), (norms.out, out), (norms.dy, dy), (norms.dx, dx), (norms.dgate, dgate), (norms.dw_pre, dwa), (norms.dw_post, dwb)):
        assert torch.isfinite(a).all() and torch.equal(a, b)
    assert float(norms.dx.float().norm()) > 0 and float(buf.dlogits.norm()) > 0


@pytest.mark.parametrize("T, d, k", [(7, 512, 4), (67, 2880, 8), (3, 16384, 2), (2000, 128, 1)])
@pytest.mark.parametrize("weighted", [False, True])
def test_post_norm_over_rows_with_unit_weights_and_without_their_sum(M, T, d, k, weighted):
    """row_of without topk_w is the unweighted sum, and the sum need not be kept: the same out and rstd."""
    g = torch.Generator("cuda").manual_seed(T + d)
    Y, x = (torch.randn(r, d, device="cuda", generator=g).to(BF) for r in (T * k + 3, T))
    w = (1 + torch.randn(d, device="cuda", generator=g) * 0.3).to(BF)
    row_of = torch.randperm(T * k + 3, device="cuda", generator=g)[:T * k].int()
    tw = torch.rand(T, k, device="cuda", generator=g) if weighted else None
    total, out, out2, rs, rs2 = (torch.full(s, float("nan"), dtype=t, device="cuda")
                                 for s, t in (((T, d), BF), ((T, d), BF), ((T, d), BF), ((T,), F32), ((T,), F32)))
    M.moe_post_norm_fwd(Y, x, w, out, rs, EPS, row_of=row_of, topk_w=tw, total=total, scale=0.7)
    want = torch.empty_like(total)
    M.moe_combine(Y, row_of, tw, k, want)
    assert torch.equal(total, want)
    v = Y[row_of.long()].view(T, k, d).double() * (1 if tw is None else tw.double().unsqueeze(2))
    # a sum of k terms in fp32, rounded to bf16
    assert ((total.double() - v.sum(1)).abs() <= 2.0**-8 * v.sum(1).abs() + 2 * k * 2.0**-24 * v.abs().sum(1)).all()
    M.moe_post_norm_fwd(Y, x, w, out2, rs2, EPS, row_of=row_of, topk_w=tw, scale=0.7)
    assert torch.equal(out, out2) and torch.equal(rs, rs2) and torch.isfinite(out).all()
    alone = torch.empty_like(out)
    M.moe_post_norm_fwd(total, x, w, alone, None, EPS, scale=0.7)
    assert torch.equal(alone, out)
