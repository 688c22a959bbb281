"""The layer's router with any number of experts, not only multiples of 8 (GPU).

Bounds: logits are fp32 sums of d products of bf16 values, off by at most (d + 2) 2^-24 of the sum of
magnitudes. The gradient products take dlogits rounded to bf16 (2^-8 of each), sum in fp32, and dx is
rounded to bf16 twice (routed part, then the sum): (d + 2) or (T + 2) 2^-24 and 2^-8 of the terms."""
import numpy as np
import pytest
import torch

from oracle import dense_oracle as D
from ragged_grouped_gemm_device_amd import workloads as W

from ._util import bf16_tensor, bf16_values

pytestmark = pytest.mark.gpu
U, H = 2.0**-24, 2.0**-8


@pytest.fixture(scope="module")
def M():
    from ragged_grouped_gemm_device_amd import moe
    moe.load()
    return moe


def _made(M, T, d, E, k, seed):
    rng = np.random.default_rng(seed)
    new = lambda *s, std=1.0: bf16_tensor(W.f32_to_bf16_bits(rng.standard_normal(s).astype(np.float32) * std))  # noqa: E731
    x, wg, dx = new(T, d), new(d, E, std=d**-0.5), new(T, d)
    base = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).cuda()
    return M.Router(T, d, E, k, 1, 0.3, 0.02), x, wg, dx, base


@pytest.mark.parametrize("T, d, E, k", [(1, 64, 1, 1), (5, 72, 3, 2), (97, 128, 4, 1), (300, 128, 12, 2), (257, 320, 60, 4),
                                        (4100, 64, 100, 6), (33, 64, 1023, 8), (300, 128, 16, 2)])
def test_router_of_any_number_of_experts(M, T, d, E, k):
    router, x, wg, dx, base = _made(M, T, d, E, k, T + E)
    dx0, dlogits = dx.clone(), base.clone()
    logits = router.project(x, wg)
    torch.cuda.synchronize()
    assert logits is router.logits and tuple(logits.shape) == (T, E) and logits.is_contiguous()
    xv, wv = bf16_values(x), bf16_values(wg)
    got = logits.cpu().numpy()
    assert (np.abs(got - xv @ wv) <= (d + 2) * U * (np.abs(xv) @ np.abs(wv)) + 2.0**-120).all()
    idx = logits.topk(k, 1).indices.to(torch.int32)
    router.losses(idx)
    router.backward(x, wg, dlogits, dx)
    torch.cuda.synchronize()
    ref = D.balance_loss(got, idx.cpu().numpy(), balance_coef=0.3, z_coef=0.02)
    assert np.array_equal(router.counts.cpu().numpy(), ref["counts"])
    assert np.allclose(router.loss.cpu().numpy(), ref["loss"], rtol=1e-4)   # its own tests hold it closer
    want = base.cpu().numpy() + ref["dlogits"]
    dl = dlogits.cpu().numpy().astype(np.float64)
    assert np.allclose(dl, want, rtol=1e-5, atol=1e-6)
    d16 = bf16_values(router.dlogits16)
    assert (np.abs(d16 - dl) <= H * np.abs(dl)).all()
    a, b = d16 @ wv.T, np.abs(d16) @ np.abs(wv).T
    full = a + bf16_values(dx0)
    bound = (E + 10) * U * (b + np.abs(bf16_values(dx0)))
    assert (np.abs(bf16_values(dx) - full) <= bound + H * (np.abs(full) + bound) + 2.0**-120).all()
    dwg = router.dwg.cpu().numpy()
    assert dwg.shape == (d, E)
    assert (np.abs(dwg - xv.T @ d16) <= (T + 2) * U * (np.abs(xv).T @ np.abs(d16)) + 2.0**-120).all()


def test_captured_router_follows_its_weights(M):
    """12 experts: new inputs and weights between the replays, against an eager router."""
    T, d, E, k = 130, 64, 12, 2
    router, x, wg, dx, base = _made(M, T, d, E, k, 3)
    eager = _made(M, T, d, E, k, 3)[0]
    dlogits, idx = base.clone(), torch.empty(T, k, dtype=torch.int32, device="cuda")
    start = dx.clone()

    def step(r, dl, to):
        dl.copy_(base)
        to.copy_(start)
        r.project(x, wg)
        r.losses(idx)
        r.backward(x, wg, dl, to)

    idx.copy_(torch.arange(T * k, device="cuda").view(T, k) % E)
    step(router, dlogits, dx)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(router, dlogits, dx)
    for rep in range(3):
        gen = torch.Generator("cuda").manual_seed(rep)
        for t in (x, wg):
            t.copy_(torch.randn(t.shape, device="cuda", generator=gen))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        dl2, dx2 = torch.empty_like(dlogits), torch.empty_like(dx)
        step(eager, dl2, dx2)
        torch.cuda.synchronize()
        assert torch.equal(dlogits, dl2) and torch.equal(dx, dx2)
        for name in ("logits", "loss", "counts", "prob", "tokens", "dwg", "dlogits16"):
            assert torch.equal(getattr(router, name), getattr(eager, name)), (rep, name)


def test_layer_with_12_experts(M):
    """Through forward and backward: the same bits as with the logits given and the router's steps by hand."""
    T, k, E, d, n = 150, 2, 12, 128, 64
    router, x, wg, _, _ = _made(M, T, d, E, k, 5)
    rng = np.random.default_rng(6)
    new = lambda *s, std=1.0: bf16_tensor(W.f32_to_bf16_bits(rng.standard_normal(s).astype(np.float32) * std))  # noqa: E731
    w1, w2, dout = new(E, d, 2 * n, std=d**-0.5), new(E, n, d, std=n**-0.5), new(T, d)
    buf, one = M.Buffers(T, k, E, d, n), M.Buffers(T, k, E, d, n)
    M.forward(buf, x, None, w1, w2, router=(router, wg))
    M.backward(buf, dout, w1, w2, router=(router, wg), x_tokens=x)
    hand = _made(M, T, d, E, k, 5)[0]
    M.forward(one, x, hand.project(x, wg), w1, w2)
    hand.losses(one.topk_idx)
    M.backward(one, dout, w1, w2, logits=hand.logits)
    hand.backward(x, wg, one.dlogits, one.dx)
    torch.cuda.synchronize()
    for name in ("out", "dx", "dlogits", "dw1", "dw2"):
        assert torch.equal(getattr(buf, name), getattr(one, name)), name
    assert torch.equal(router.dwg, hand.dwg) and torch.equal(router.loss, hand.loss)
