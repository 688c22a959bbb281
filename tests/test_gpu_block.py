"""A whole residual block: norm, router with scores, bias and groups, routed experts (bf16 or 4-bit), shared expert,
combination with the second norm, gate and scaled residual, forward and backward, against the oracles;
captured into a graph; on two streams (GPU).

Bounds: max-abs-normalised 2e-2, the routed path's own (its parts round to bf16 in between)."""
import numpy as np
import pytest
import torch

from oracle import block_oracle as B
from oracle import dense_oracle as D
from oracle import moe_oracle as O
from ragged_grouped_gemm_device_amd import workloads as W

from ._util import bf16_tensor, bf16_values, f32_tensor, rel_err

pytestmark = pytest.mark.gpu
SCALE = 0.5


@pytest.fixture(scope="module")
def M():
    from ragged_grouped_gemm_device_amd import moe
    moe.load()
    return moe


class Block:
    def __init__(self, M, wl, cols, shared=True, act="swiglu", seed=0, **how):
        self.M, self.wl, self.act = M, wl, act
        inp = W.make_inputs(wl)
        rng = np.random.default_rng(wl.seed + seed)
        if act not in D.GATED:
            inp["w1"] = inp["w1"][:, :, :wl.n]
        self.t = t = {k: bf16_tensor(inp[k]) for k in ("x", "w1", "w2", "dout")}
        ns = 96
        n1 = 2 * ns if act in D.GATED else ns
        new = lambda *shape, std=1.0, mean=0.0: bf16_tensor(W.f32_to_bf16_bits(  # noqa: E731
            (rng.standard_normal(shape) * std + mean).astype(np.float32)))
        t.update(wg=new(wl.d, wl.E, std=wl.d**-0.5), s1=new(wl.d, n1, std=wl.d**-0.5), s2=new(ns, wl.d, std=ns**-0.5),
                 wa=new(wl.d, std=0.2, mean=1.0), wb=new(wl.d, std=0.2, mean=1.0))
        if cols:
            t["gate"] = new(wl.T, cols)
        self.bias = (rng.standard_normal(wl.E) * 0.05).astype(np.float32)
        self.how = dict(groups=4, topk_groups=2, group_top=2, renorm=True, scale=1.5) | how
        self.routing = M.Routing(M.MOE_SCORE_SIGMOID, f32_tensor(self.bias), **self.how)
        self.buf = M.Buffers(wl.T, wl.k, wl.E, wl.d, wl.n, gated=act in D.GATED)
        self.router = M.Router(wl.T, wl.d, wl.E, wl.k, balance_coef=0.0, z_coef=0.0)
        self.shared = M.SharedExpert(wl.T, wl.d, ns, D.ACTS.index(act), ckpt8=False) if shared else None
        self.norms = M.BlockNorms(wl.T, wl.d, cols, M.MOE_GATE_SIGMOID, SCALE)

    def kw(self):
        t = self.t
        return dict(router=(self.router, t["wg"]), shared=None if self.shared is None else (self.shared, t["s1"], t["s2"]),
                    routing=self.routing, norms=(self.norms, t["wa"], t["wb"], t.get("gate")), act=D.ACTS.index(self.act))

    def forward(self, **more):
        self.M.forward(self.buf, self.t["x"], None, self.t["w1"], self.t["w2"], **self.kw(), **more)

    def backward(self, gather=False):
        x = {"x": self.t["x"]} if gather else {"x_tokens": self.t["x"]}
        self.M.backward(self.buf, self.t["dout"], self.t["w1"], self.t["w2"], **self.kw(), **x)

    def results(self):
        n, r = self.norms, {}
        r.update(out=n.out, dx=n.dx, dwa=n.dw_pre, dwb=n.dw_post, dw1=self.buf.dw1, dw2=self.buf.dw2, dlogits=self.buf.dlogits,
                 dwg=self.router.dwg)
        if n.dgate is not None:
            r["dgate"] = n.dgate
        if self.shared is not None:
            r.update(ds1=self.shared.dw1, ds2=self.shared.dw2)
        return r

    def oracle(self):
        wl, act = self.wl, self.act
        v = {k: bf16_values(x) for k, x in self.t.items()}
        h = B.norm(v["x"], v["wa"], 1e-6)[0]
        logits = self.router.logits.cpu().numpy()
        assert rel_err(logits, h @ v["wg"]) <= 1e-2
        h = bf16_values(self.norms.y)
        how = self.how
        idx, w = B.route_scores(logits, self.bias, "sigmoid", wl.k, how["groups"], how["topk_groups"], 2, True, how["scale"])
        assert np.array_equal(self.buf.topk_idx.cpu().numpy(), idx)
        counts, offsets, row_of, src_of = O.layout(idx, wl.E, self.buf.M_cap)
        xp = O.permute(h, row_of, wl.k, self.buf.M_cap)
        H, _, Y = O.mlp_forward(xp, v["w1"], v["w2"], counts, offsets, act=act)
        y = O.combine(Y, row_of, wl.k, w)
        z = h @ v["s1"]
        a = D.act_forward(z, act)
        if self.shared is not None:
            y = y + a @ v["s2"]
        gate = v.get("gate")
        out, _ = B.post_norm(y, v["x"], v["wb"], 1e-6, gate, True, SCALE)
        dy, dgate, dwb = B.post_norm_bwd(v["dout"], y, v["wb"], 1e-6, gate, True, SCALE)
        b = O.mlp_backward(xp, v["w1"], v["w2"], H, Y, dy, w, counts, offsets, row_of, src_of, wl.k, act=act)
        dlog = B.route_scores_bwd(logits, self.bias, idx, b["dS"], "sigmoid", True, how["scale"])
        dh = b["dx"] + dlog @ v["wg"].T
        r = {"out": out, "dgate": dgate, "dwb": dwb, "dw1": b["dW1"], "dw2": b["dW2"], "dlogits": dlog, "dwg": h.T @ dlog}
        if self.shared is not None:
            dz = D.act_backward(dy @ v["s2"].T, z, act)
            dh = dh + dz @ v["s1"].T
            r.update(ds1=h.T @ dz, ds2=a.T @ dy)
        dx, r["dwa"] = B.norm_bwd(dh, v["x"], v["wa"], 1e-6)
        r["dx"] = dx + v["dout"]
        return r


@pytest.mark.parametrize("T, k, E, d, n, cols, shared, act, gather", [
    (256, 2, 8, 128, 64, 128, True, "swiglu", False), (97, 3, 16, 192, 128, 1, False, "geglu", False),
    (1, 2, 8, 64, 64, 0, False, "swiglu", False), (300, 4, 32, 320, 64, 320, False, "swiglu", True),
    (130, 1, 12, 64, 64, 1, True, "srelu", True),
])
def test_block_against_the_oracles(M, T, k, E, d, n, cols, shared, act, gather):
    b = Block(M, W.small("block", T, k, E, d, n, seed=T + E), cols, shared, act)
    b.forward(gather=gather)
    b.backward(gather)
    torch.cuda.synchronize()
    ref = b.oracle()
    for key, got in b.results().items():
        assert rel_err(got.float().cpu().numpy(), ref[key]) <= 2e-2, key


@pytest.mark.parametrize("form", [0, 1, 2])
@pytest.mark.parametrize("T, k, E, d, n, act", [(1, 2, 8, 128, 64, "swiglu"), (40, 4, 16, 192, 96, "geglu"), (300, 2, 8, 320, 128, "swiglu"),
                                                (600, 2, 4, 256, 64, "srelu")])
def test_served_on_4_bit_weights(M, form, T, k, E, d, n, act):
    """The block's output on 4-bit weights is the oracle's on the values that the codes stand for; rows that are
    quantized on the way carry the format's own error as well (its relative 2-norm: below 2^-3 for E2M1's
    half step of a quarter of a value at most, a rounding of each value by 2^-2 / sqrt(3) on average at most; 2^-4 for
    E4M3), over two products."""
    wl = W.small("served", T, k, E, d, 64 if n == 96 else n, seed=T)
    b = Block(M, wl, 1, False, act)
    four = M.Experts4(T, k, E, d, wl.n, D.ACTS.index(act), form)
    four.load(b.t["w1"], b.t["w2"])
    b.forward(experts4=four)
    torch.cuda.synchronize()
    assert b.buf.served
    with pytest.raises(ValueError, match="4-bit"):
        b.backward()
    v = {key: bf16_values(x) for key, x in b.t.items()}
    w1 = B.dequant_mxfp4(four.w1_q.cpu().numpy(), four.w1_s.cpu().numpy())
    w2 = B.dequant_mxfp4(four.w2_q.cpu().numpy(), four.w2_s.cpu().numpy())
    h = bf16_values(b.norms.y)
    idx, w = b.buf.topk_idx.cpu().numpy(), b.buf.topk_w.double().cpu().numpy()
    counts, offsets, row_of, src_of = O.layout(idx, E, b.buf.M_cap)
    xp = O.permute(h, row_of, k, b.buf.M_cap)
    Y = np.nan_to_num(B.grouped_linear(np.nan_to_num(B.grouped_linear(xp, w1, offsets, counts, act)), w2, offsets, counts))
    y = O.combine(Y, row_of, k, w, rounding=False)
    got = bf16_values(b.buf.out)
    off = np.linalg.norm(got - y) / np.linalg.norm(y)
    assert off <= (1e-2, 2 * 2.0**-4, 2 * 2.0**-2 / 3**0.5 + 2.0**-4)[form], off
    out, _ = B.post_norm(got, v["x"], v["wb"], 1e-6, v["gate"], True, SCALE)
    assert rel_err(bf16_values(b.norms.out), out) <= 2e-2


def test_block_captured_and_replayed(M):
    wl = W.small("graph", 200, 2, 8, 128, 64, seed=5)
    one, two = Block(M, wl, 128), Block(M, wl, 128)
    one.forward()
    one.backward()
    torch.cuda.synchronize()
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            one.forward()
            one.backward()
    for rep in range(3):
        for key in ("x", "dout", "gate"):
            one.t[key].copy_(torch.randn(one.t[key].shape, device="cuda", generator=torch.Generator("cuda").manual_seed(rep)))
            two.t[key].copy_(one.t[key])
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        two.forward()
        two.backward()
        torch.cuda.synchronize()
        for (key, a), b in zip(one.results().items(), two.results().values()):
            assert torch.equal(a, b), (rep, key)


def test_serving_graph_of_a_token_at_a_time(M):
    """Decode steps replayed from a graph, each with its own routing."""
    wl = W.small("decode", 4, 2, 8, 128, 64, seed=8)
    one, two = Block(M, wl, 0, False), Block(M, wl, 0, False)
    fours = [M.Experts4(4, 2, 8, 128, 64) for _ in range(2)]
    for b, f in zip((one, two), fours):
        f.load(b.t["w1"], b.t["w2"])
        b.forward(experts4=f)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        one.forward(experts4=fours[0])
    for rep in range(4):
        x = torch.randn(4, 128, device="cuda", generator=torch.Generator("cuda").manual_seed(rep)).bfloat16()
        one.t["x"].copy_(x)
        two.t["x"].copy_(x)
        torch.cuda.synchronize()
        g.replay()
        two.forward(experts4=fours[1])
        torch.cuda.synchronize()
        assert torch.equal(one.norms.out, two.norms.out) and torch.equal(one.buf.topk_idx, two.buf.topk_idx), rep


def test_two_streams(M):
    wl = W.small("streams", 128, 2, 8, 128, 64, seed=6)
    blocks = [Block(M, wl, 1), Block(M, wl, 1)]
    blocks[0].forward()
    blocks[0].backward()
    torch.cuda.synchronize()
    want = {key: v.clone() for key, v in blocks[0].results().items()}
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for st, b in zip(streams, blocks):
            with torch.cuda.stream(st):
                b.forward()
                b.backward()
    torch.cuda.synchronize()
    for b in blocks:
        for key, v in b.results().items():
            assert torch.equal(v, want[key]), key
