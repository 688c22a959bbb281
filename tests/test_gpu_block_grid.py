"""Norms and the router's gradient of more tokens than one launch has room for: a workgroup's share of them each, they
would be 2^32 threads and more, which is cut off without an error (GPU). The rows repeat a block of 4096, so that
every result is that of the block."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
BLOCK = 4096


@pytest.fixture(scope="module")
def M():
    from ragged_grouped_gemm_device_amd import moe
    moe.load()
    return moe


def tiled(block, T):
    return block.repeat(-(-T // BLOCK), *[1] * (block.dim() - 1))[:T]


def same(got, block):
    T = got.shape[0]
    step = BLOCK << 8
    for t in range(0, T, step):
        part = got[t:t + step]
        assert torch.equal(part, tiled(block, part.shape[0])), t


@pytest.mark.parametrize("T, d", [((1 << 26) + 5, 8), ((1 << 24) + 5, 1032)])
def test_norm(M, T, d):
    g = torch.Generator("cuda").manual_seed(d)
    x, w = torch.randn(BLOCK, d, device="cuda", generator=g).to(BF), torch.randn(d, device="cuda", generator=g).to(BF)
    y, rstd = torch.empty_like(x), torch.empty(BLOCK, device="cuda")
    M.moe_norm_fwd(x, w, y, rstd)
    big, r = torch.full((T, d), float("nan"), dtype=BF, device="cuda"), torch.full((T,), float("nan"), device="cuda")
    M.moe_norm_fwd(tiled(x, T), w, big, r)
    same(big, y)
    same(r, rstd)


@pytest.mark.parametrize("rows", [False, True])
def test_norm_with_residual_and_post_norm(M, rows):
    T, d = (1 << 26) + 5, 8
    g = torch.Generator("cuda").manual_seed(7)
    x, v, gate = (torch.randn(BLOCK, d, device="cuda", generator=g).to(BF) for _ in range(3))
    w = torch.randn(d, device="cuda", generator=g).to(BF)
    gate = gate if rows else gate[:, :1].contiguous()
    topk_w = torch.rand(BLOCK, 2, device="cuda", generator=g)
    row_of = torch.randint(0, BLOCK, (2 * BLOCK,), device="cuda", generator=g, dtype=I32)
    new = lambda n, *s, t=BF: torch.full((n, *s), float("nan"), dtype=t, device="cuda")  # noqa: E731

    def run(n, t):
        if not rows:
            total, y, r = new(n, d), new(n, d), new(n, t=F32)
            M.moe_norm_fwd(t(x), w, y, r, residual=t(v), total=total)
            out, r2 = new(n, d), new(n, t=F32)
            M.moe_post_norm_fwd(t(v), t(x), w, out, r2, gate=t(gate), scale=0.5)
            return total, y, r, out, r2
        total, out, r = new(n, d), new(n, d), new(n, t=F32)
        at = t(row_of.view(BLOCK, 2)).reshape(-1)
        M.moe_post_norm_fwd(v, t(x), w, out, r, gate=t(gate), gate_act=M.MOE_GATE_SIGMOID, row_of=at, topk_w=t(topk_w), total=total)
        return total, out, r

    for big, block in zip(run(T, lambda a: tiled(a, T)), run(BLOCK, lambda a: a)):
        assert torch.isfinite(block).all()
        same(big, block)


@pytest.mark.parametrize("T, E, k", [((1 << 28) + 5, 4, 2), ((1 << 26) + 5, 20, 17)])
def test_router_gradient(M, T, E, k):
    g = torch.Generator("cuda").manual_seed(E)
    lg, ds = torch.randn(BLOCK, E, device="cuda", generator=g), torch.randn(BLOCK, k, device="cuda", generator=g)
    idx = torch.rand(BLOCK, E, device="cuda", generator=g).topk(k, 1).indices.int()
    for score, renorm in ((M.MOE_SCORE_SIGMOID, True), (M.MOE_SCORE_SOFTMAX, False)):
        how = M.Routing(score, renorm=renorm)
        block, big = torch.empty_like(lg), torch.full((T, E), float("nan"), device="cuda")
        M.moe_route_scores_bwd(lg, idx, ds, block, how)
        M.moe_route_scores_bwd(tiled(lg, T), tiled(idx, T), tiled(ds, T), big, how)
        same(big, block)
