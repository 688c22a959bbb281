"""The router with scores, bias and groups against the fp64 oracle (GPU). Choices and layout are equal;
weights and gradients are fp32 results of at most 16 roundings each: 16 * 2^-24 relative, and for the
gradients of the largest term (differences of terms cancel)."""
import numpy as np
import pytest
import torch

from oracle import block_oracle as B
from oracle import moe_oracle as O

from ._util import f32_tensor

pytestmark = pytest.mark.gpu
TOL = 16 * 2.0**-24
I32, F32 = torch.int32, torch.float32


@pytest.fixture(scope="module")
def M():
    from ragged_grouped_gemm_device_amd import moe
    moe.load()
    return moe


class Call:
    """One routing with its own buffers, prefilled with what no result is."""

    def __init__(self, M, lg, bias, k, score="sigmoid", groups=1, kept=1, top=2, renorm=True, scale=1.0, device_logits=None):
        T, E = lg.shape
        self.lg = f32_tensor(lg) if device_logits is None else device_logits
        how = dict(groups=groups, topk_groups=kept, group_top=top, renorm=renorm, scale=scale)
        self.M, self.k, self.cap = M, k, M.moe_capacity_rows(T, k, E)
        self.routing = M.Routing(M.MOE_SCORE_SIGMOID if score == "sigmoid" else M.MOE_SCORE_SOFTMAX,
                                 None if bias is None else f32_tensor(bias), **how)
        full = lambda *s, t=I32: torch.full(s, -7, dtype=t, device="cuda")  # noqa: E731
        self.idx, self.w, self.counts, self.offsets = full(T, k), full(T, k, t=F32), full(E), full(E + 1)
        self.row_of, self.src_of, self.err = full(T * k), full(self.cap), torch.zeros(1, dtype=I32, device="cuda")
        self.ws = torch.full((max(16, M.moe_route_scores_workspace_bytes(T, k, E)),), 77, dtype=torch.uint8, device="cuda")
        self.dlogits = torch.full((T, E), float("nan"), device="cuda")

    def run(self):
        self.M.moe_route_scores(self.lg, self.k, self.idx, self.w, self.counts, self.offsets, self.row_of, self.src_of, self.err,
                                self.ws, self.routing)
        return self

    def bwd(self, ds):
        self.M.moe_route_scores_bwd(self.lg, self.idx, ds, self.dlogits, self.routing)
        return self


def check(M, lg, bias, k, score="sigmoid", groups=1, kept=1, top=2, renorm=True, scale=1.0, bwd=True):
    c = Call(M, lg, bias, k, score, groups, kept, top, renorm, scale).run()
    idx, w = B.route_scores(lg, bias, score, k, groups, kept, top, renorm, scale)
    got = c.idx.cpu().numpy()
    assert np.array_equal(got, idx), np.flatnonzero((got != idx).any(1))[:5]
    counts, offsets, row_of, src_of = O.layout(idx, lg.shape[1], c.cap)
    for name, want in (("counts", counts), ("offsets", offsets), ("row_of", row_of), ("src_of", src_of)):
        assert np.array_equal(getattr(c, name).cpu().numpy(), want), name
    np.testing.assert_allclose(c.w.cpu().numpy(), w, rtol=TOL, atol=abs(scale) * 2.0**-126)
    assert int(c.err) == (0 if np.isfinite(lg).all() else M.MOE_ERRBIT_NONFINITE_LOGIT)
    if bwd:
        ds = np.random.default_rng(1).standard_normal(idx.shape).astype(np.float32)
        c.bwd(f32_tensor(ds))
        ref = B.route_scores_bwd(lg, bias, idx, ds, score, renorm, scale)
        most = np.abs(w).max(1, keepdims=True) * np.abs(ds).max(1, keepdims=True)  # every term is within it
        assert (np.abs(c.dlogits.cpu().numpy() - ref) <= 2 * TOL * most + 1e-37).all()
    return c


def logits(T, E, seed=0, spread=1.0):
    return (np.random.default_rng(seed).standard_normal((T, E)) * spread).astype(np.float32)


@pytest.mark.parametrize("T, E, k, groups, kept", [
    (1, 1, 1, 1, 1), (1, 256, 8, 8, 4), (5, 3, 2, 1, 1), (17, 12, 4, 3, 2), (63, 64, 8, 8, 3), (64, 65, 5, 5, 2), (100, 128, 16, 4, 2),
    (130, 160, 6, 8, 3), (33, 256, 8, 8, 4), (20, 257, 8, 1, 1), (20, 256, 17, 16, 9), (9, 512, 64, 64, 8), (12, 1024, 8, 32, 5),
    (7, 1000, 33, 8, 8), (40, 48, 3, 48, 5), (21, 60, 60, 2, 2), (300, 2, 1, 2, 1),
])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_against_the_oracle(M, T, E, k, groups, kept, score):
    lg = logits(T, E, T + E)
    bias = (np.random.default_rng(E).standard_normal(E) * 0.1).astype(np.float32)
    check(M, lg, bias, k, score, groups, kept, 2, True, 2.5)
    check(M, lg, None, k, score, groups, kept, 1, False, 1.0)
    check(M, lg, None, k, score, groups, kept, 2, False, -0.5, bwd=False)
    check(M, lg, bias, k, score, groups, kept, 1, False, 1.0, bwd=False)


@pytest.mark.parametrize("T, E, k", [(3000, 32, 4), (2500, 256, 8)])
def test_many_tokens(M, T, E, k):
    """Several chunks; the choice of every token, those near a border among them."""
    check(M, logits(T, E, 7), (np.random.default_rng(3).standard_normal(E) * 0.05).astype(np.float32), k, "sigmoid", 4, 2)


def test_layout_over_many_chunks(M):
    """Past the two-kernel form: the layout of the choices that the call itself made."""
    T, E, k = 40000, 256, 8
    lg = logits(T, E, 11)
    c = Call(M, lg, None, k, groups=8, kept=4, top=1).run()
    idx = c.idx.cpu().numpy()
    for name, want in zip(("counts", "offsets", "row_of", "src_of"), O.layout(idx, E, c.cap)):
        assert np.array_equal(getattr(c, name).cpu().numpy(), want), name
    some = np.r_[0:50, T - 50:T]
    assert np.array_equal(idx[some], B.route_scores(lg[some], None, "sigmoid", k, 8, 4, 1)[0])


def test_values_that_lie_close(M):
    """Choice values that fp32 scores cannot order (the bias makes up for the score to a part in 2^30),
    equal ones, and equal values of different scores: the oracle's order, lower index first."""
    rng = np.random.default_rng(5)
    E, k = 64, 8
    lg = logits(200, E, 6)
    for score in ("sigmoid", "softmax"):
        s = np.array([B.scores(r.astype(np.float64), score) for r in lg])
        for t in range(0, 200, 4):
            # this token's scores plus the bias are nearly one value
            bias = (0.75 - s[t] + rng.integers(-3, 4, E) * 2.0**-30).astype(np.float32)
            sub = lg[t:t + 4]
            check(M, sub, bias, k, score, 8, 3, 2, bwd=False)
            check(M, sub, bias, k, score, bwd=False)
    same = np.zeros((9, E), np.float32)
    check(M, same, np.zeros(E, np.float32), k, groups=8, kept=2)
    check(M, same, None, k, groups=8, kept=2, top=1)
    twice = np.repeat(logits(30, E // 2, 8), 2, axis=1)
    check(M, twice, np.zeros(E, np.float32), k, groups=4, kept=2)
    check(M, twice, None, k, "softmax", groups=4, kept=2, top=1)


def test_large_and_small_scores(M):
    """Saturated scores, ones that underflow (renormalised weights keep their ratios), huge biases."""
    lg = logits(40, 32, 9, 30.0)
    check(M, lg, None, 4)
    check(M, lg, None, 4, "softmax", renorm=True)
    check(M, lg - 150, None, 4, groups=4, kept=2, top=1)
    check(M, lg * 1e30, None, 4, "softmax", renorm=True)
    bias = np.linspace(-1e6, 1e6, 32).astype(np.float32)
    check(M, logits(40, 32, 10), bias, 4, groups=4, kept=2)
    check(M, logits(40, 32, 10), (bias * 1e30).astype(np.float32), 4)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E, k, groups, kept", [(16, 4, 1, 1), (64, 6, 8, 2), (512, 20, 4, 1)])
def test_experts_out_of_service_and_bad_logits(M, score, E, k, groups, kept):
    """Biases that are not finite and logits that are not, down to nothing left: in range, lowest index first,
    weight and gradient 0."""
    rng = np.random.default_rng(E)
    for share in (0.1, 0.9, 1.0):
        lg = logits(30, E, E + 1)
        bias = (rng.standard_normal(E) * 0.1).astype(np.float32)
        bias[rng.random(E) < share] = -np.inf
        for renorm in (False, True):
            check(M, lg, bias, k, score, groups, kept, 2, renorm)
        for value in (np.nan, np.inf, -np.inf):
            lg[rng.random(lg.shape) < share / 3] = value
        check(M, lg, None, k, score, groups, kept, 1)
        check(M, lg, bias, k, score, groups, kept, 2)
    bias[:] = [np.nan, np.inf] * (E // 2)
    check(M, logits(5, E), bias, k, score, groups, kept)


def test_logits_at_any_4_bytes(M):
    base = torch.zeros(33 * 64 + 1, device="cuda")
    lg = logits(33, 64, 4)
    base[1:].copy_(f32_tensor(lg).reshape(-1))
    c = Call(M, lg, None, 4, device_logits=base[1:].view(33, 64)).run()
    assert np.array_equal(c.idx.cpu().numpy(), B.route_scores(lg, None, "sigmoid", 4)[0])
    ds = torch.ones(33, 4, device="cuda")
    a = c.bwd(ds).dlogits.clone()
    d = Call(M, lg, None, 4).run().bwd(ds)
    assert torch.equal(a, d.dlogits) and torch.equal(c.w, d.w)


def test_backward_leaves_out_slots_past_the_experts(M):
    """Choices that no forward made (out of range) reach no memory and have no gradient."""
    lg = logits(6, 8)
    c = Call(M, lg, None, 2, renorm=False).run()
    c.idx[2, 1], c.idx[3, 0] = 8, -1
    c.bwd(torch.ones(6, 2, device="cuda"))
    got = c.dlogits.cpu().numpy()
    assert np.isfinite(got).all() and (got[2] != 0).sum() == 1 and (got[3] != 0).sum() == 1


def test_captured_and_on_two_streams(M):
    T, E, k = 900, 128, 6
    calls = [Call(M, logits(T, E, s), np.linspace(-.1, .1, E).astype(np.float32), k, groups=4, kept=2) for s in (1, 2)]
    ds = torch.randn(T, k, device="cuda")
    for c in calls:
        c.run().bwd(ds)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        calls[0].run().bwd(ds)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for rep in range(3):
        lg = logits(T, E, 20 + rep)
        want = Call(M, lg, np.linspace(-.1, .1, E).astype(np.float32), k, groups=4, kept=2).run().bwd(ds)
        for c in calls:
            c.lg.copy_(f32_tensor(lg))
        torch.cuda.synchronize()
        with torch.cuda.stream(streams[0]):
            g.replay()
        with torch.cuda.stream(streams[1]):
            calls[1].run().bwd(ds)
        torch.cuda.synchronize()
        for c in calls:
            for name in ("idx", "w", "counts", "offsets", "row_of", "src_of", "dlogits"):
                assert torch.equal(getattr(c, name), getattr(want, name)), (rep, name)
