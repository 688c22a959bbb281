"""The whole layer: router projection, routing, router losses, routed experts, shared expert,
forward and backward, against the oracles; captured into a graph; 8-bit checkpoints (GPU).

Bounds: max-abs-normalised 2e-2, the routed path's own (its parts round to bf16 in between);
an 8-bit checkpoint moves each kept value by at most 2^-4 of it, independently, so a gradient
made of it moves by about 2^-4 / sqrt(3) in norm at worst: 6e-2 there."""
import numpy as np
import pytest
import torch

from oracle import dense_oracle as D
from oracle import moe_oracle as O
from ragged_grouped_gemm_device_amd import workloads as W

from ._util import bf16_tensor, bf16_values, rel_err

pytestmark = pytest.mark.gpu
CB, CZ = 0.05, 0.01


@pytest.fixture(scope="module")
def M():
    from ragged_grouped_gemm_device_amd import moe
    moe.load()
    return moe


def _layer(M, wl, act="swiglu", ckpt8=False, x8=False, ns=96, seqs=None):
    inp = W.make_inputs(wl)
    rng = np.random.default_rng(wl.seed)
    t = {k: bf16_tensor(inp[k]) for k in ("x", "w1", "w2", "dout")}
    n1 = 2 * ns if act in D.GATED else ns
    for name, shape, std in (("wg", (wl.d, wl.E), wl.d**-0.5), ("s1", (wl.d, n1), wl.d**-0.5), ("s2", (ns, wl.d), ns**-0.5)):
        t[name] = bf16_tensor(W.f32_to_bf16_bits(rng.standard_normal(shape).astype(np.float32) * std))
    buf = M.Buffers(wl.T, wl.k, wl.E, wl.d, wl.n, ckpt8=ckpt8)
    S = 1 if seqs is None else len(seqs) - 1
    router = M.Router(wl.T, wl.d, wl.E, wl.k, S, CB, CZ)
    if seqs is not None:
        router.seq_offsets = torch.tensor(seqs, dtype=torch.int32, device="cuda")
        router.valid = torch.from_numpy((rng.random(wl.T) < 0.9).astype(np.uint8)).cuda()
    shared = M.SharedExpert(wl.T, wl.d, ns, D.ACTS.index(act), ckpt8=ckpt8, x8=x8)
    return t, buf, router, shared


def _step(M, t, buf, router, shared, x8=False):
    r, s = (router, t["wg"]), (shared, t["s1"], t["s2"])
    M.forward(buf, t["x"], None, t["w1"], t["w2"], router=r, shared=s)
    M.backward(buf, t["dout"], t["w1"], t["w2"], router=r, shared=s, x_tokens=t["x"])


def _results(buf, router, shared):
    return {"out": buf.out, "dx": buf.dx, "dw1": buf.dw1, "dw2": buf.dw2, "dlogits": buf.dlogits, "loss": router.loss,
            "dwg": router.dwg, "ds1": shared.dw1, "ds2": shared.dw2}


def _oracle(t, buf, router, act, wl, z=None):
    v = {k: bf16_values(x) for k, x in t.items()}
    logits = router.logits.cpu().numpy()
    assert rel_err(logits, v["x"] @ v["wg"]) <= 1e-5
    f = O.forward(v["x"], logits, v["w1"], v["w2"], wl.k)
    assert np.array_equal(buf.topk_idx.cpu().numpy(), f["topk_idx"])
    b = O.mlp_backward(f["x_perm"], v["w1"], v["w2"], f["H"], f["Y"], v["dout"], f["topk_w"], f["counts"], f["offsets"],
                       f["row_of"], f["src_of"], wl.k)
    valid = None if router.valid is None else router.valid.cpu().numpy()
    offs = None if router.seq_offsets is None else router.seq_offsets.cpu().numpy()
    bal = D.balance_loss(logits, f["topk_idx"], valid, offs, CB, CZ)
    dlog = O.route_backward(logits, f["topk_idx"], b["dS"]) + bal["dlogits"]
    z0 = v["x"] @ v["s1"]
    a = D.act_forward(z0, act)
    da = v["dout"] @ v["s2"].T
    dz = D.act_backward(da, z0, act)
    return {"out": f["out"] + a @ v["s2"], "dx": b["dx"] + dz @ v["s1"].T + dlog @ v["wg"].T, "dw1": b["dW1"],
            "dw2": b["dW2"], "dlogits": dlog, "loss": bal["loss"], "dwg": v["x"].T @ dlog, "ds1": v["x"].T @ dz,
            "ds2": a.T @ v["dout"]}


@pytest.mark.parametrize("act, T, k, E, d, n, ns, seqs", [
    ("swiglu", 256, 2, 8, 128, 64, 96, None),
    ("geglu", 97, 1, 16, 192, 128, 32, [0, 30, 30, 80]),
    ("srelu", 1, 1, 8, 64, 64, 40, None),
    ("gelu", 600, 4, 32, 320, 64, 1032, [0, 100, 600]),
])
def test_layer_against_the_oracles(M, act, T, k, E, d, n, ns, seqs):
    wl = W.small("layer", T, k, E, d, n, seed=T + E)
    t, buf, router, shared = _layer(M, wl, act, ns=ns, seqs=seqs)
    _step(M, t, buf, router, shared)
    torch.cuda.synchronize()
    ref = _oracle(t, buf, router, act, wl)
    for key, got in _results(buf, router, shared).items():
        assert rel_err(got.float().cpu().numpy(), ref[key]) <= 2e-2, key


@pytest.mark.parametrize("x8", [False, True])
def test_layer_with_8_bit_checkpoints(M, x8):
    wl = W.small("ckpt", 300, 2, 8, 128, 64, seed=77)
    t, buf, router, shared = _layer(M, wl, ckpt8=True, x8=x8)
    M.forward(buf, t["x"], None, t["w1"], t["w2"], router=(router, t["wg"]), shared=(shared, t["s1"], t["s2"]))
    buf.h.fill_(float("nan"))                  # scratch between forward and backward
    M.backward(buf, t["dout"], t["w1"], t["w2"], router=(router, t["wg"]), shared=(shared, t["s1"], t["s2"]), x_tokens=t["x"])
    torch.cuda.synchronize()
    ref = _oracle(t, buf, router, "swiglu", wl)
    for key, got in _results(buf, router, shared).items():
        got = got.float().cpu().numpy()
        if key in ("out", "loss"):
            assert rel_err(got, ref[key]) <= 2e-2, key
        else:
            assert np.linalg.norm(got - ref[key]) <= 6e-2 * np.linalg.norm(ref[key]), key


def test_layer_captured_and_replayed(M):
    """A captured step equals the eager one, over replays with changed inputs and eager work between."""
    wl = W.small("graph", 200, 2, 8, 128, 64, seed=5)
    t, buf, router, shared = _layer(M, wl, ckpt8=True, seqs=[0, 50, 200])
    _step(M, t, buf, router, shared)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            _step(M, t, buf, router, shared)
    t2, buf2, router2, shared2 = _layer(M, wl, ckpt8=True, seqs=[0, 50, 200])
    router2.valid = router.valid
    for rep in range(3):
        for key in ("x", "dout"):
            t[key].copy_(torch.randn(t[key].shape, device="cuda", generator=torch.Generator("cuda").manual_seed(rep)))
            t2[key].copy_(t[key])
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        _step(M, t2, buf2, router2, shared2)
        torch.cuda.synchronize()
        for (key, a), b in zip(_results(buf, router, shared).items(), _results(buf2, router2, shared2).values()):
            assert torch.equal(a, b), (rep, key)


def test_two_streams_with_their_own_workspaces(M):
    wl = W.small("streams", 128, 2, 8, 128, 64, seed=6)
    one, two = _layer(M, wl), _layer(M, wl)
    _step(M, *one)
    torch.cuda.synchronize()
    want = {key: v.clone() for key, v in _results(*one[1:]).items()}
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for st, layer in zip(streams, (one, two)):
            with torch.cuda.stream(st):
                _step(M, *layer)
    torch.cuda.synchronize()
    for layer in (one, two):
        for key, v in _results(*layer[1:]).items():
            assert torch.equal(v, want[key]), key
