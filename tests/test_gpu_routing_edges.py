"""The router with scores at the ends of fp32's range, with gradients that are not finite, and with choices that
few lanes or many candidates hold (GPU), against the fp64 oracle; tolerances as in test_gpu_routing.py."""
import numpy as np
import pytest
import torch

from oracle import block_oracle as B

from ._util import f32_tensor
from .test_gpu_routing import M, TOL, Call, check, logits  # noqa: F401

pytestmark = pytest.mark.gpu
MOST = np.float32(np.finfo(np.float32).max)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E, k", [(64, 5), (512, 20)])
@pytest.mark.parametrize("renorm", [False, True])
def test_logits_whose_difference_is_past_fp32(M, score, E, k, renorm):
    """Chosen logits at both ends of the range: the far ones weigh 0, the others what they weigh without them."""
    rng = np.random.default_rng(E)
    lg = np.full((40, E), -MOST, np.float32) * rng.uniform(0.9, 1, (40, E)).astype(np.float32)
    for t in range(40):
        lg[t, rng.permutation(E)[:k - 2]] = MOST * np.float32(1 - 2.0**-20 * (t % 3))
    check(M, lg, None, k, score, renorm=renorm)
    bias = np.zeros(E, np.float32)
    check(M, lg, bias, k, score, renorm=renorm)


@pytest.mark.parametrize("score, renorm", [("sigmoid", True), ("sigmoid", False), ("softmax", True), ("softmax", False)])
@pytest.mark.parametrize("E, k", [(16, 4), (512, 20)])
def test_a_gradient_of_an_expert_without_weight(M, score, renorm, E, k):
    """Slots that weigh 0 for want of a finite logit or bias have no part in the gradient, whatever dL/dtopk_w says
    there: an expert out of service may well give an infinity or a NaN."""
    rng = np.random.default_rng(k)
    lg = logits(30, E, E)
    bias = np.full(E, -np.inf, np.float32)
    bias[rng.permutation(E)[:k // 2]] = 0.1
    lg[5, :] = np.nan   # nothing left at all
    c = Call(M, lg, bias, k, score, renorm=renorm).run()
    idx = c.idx.cpu().numpy()
    ds = rng.standard_normal(idx.shape).astype(np.float32)
    away = ~(np.isfinite(np.take_along_axis(lg, idx, 1)) & np.isfinite(bias[idx]))
    assert away.any() and not away.all()
    zero = np.where(away, np.float32(0), ds)
    want = c.bwd(f32_tensor(zero)).dlogits.clone()
    ref = B.route_scores_bwd(lg, bias, idx, zero, score, renorm)
    most = np.abs(c.w.cpu().numpy()).max(1, keepdims=True) * np.abs(zero).max(1, keepdims=True)
    assert (np.abs(want.cpu().numpy() - ref) <= 2 * TOL * most + 1e-37).all()
    for bad in (np.nan, np.inf, -np.inf):
        assert torch.equal(c.bwd(f32_tensor(np.where(away, np.float32(bad), ds))).dlogits, want), bad


@pytest.mark.parametrize("E, k", [(256, 4), (320, 20)])
def test_group_values_past_fp32(M, E, k):
    """Sums of two biases that fp32 does not hold, at both ends: the groups' order is that of the exact sums."""
    size = E // 8
    rng = np.random.default_rng(E)
    big = rng.permutation(np.linspace(1e38, 1.5e38, E)).astype(np.float32)
    for g in range(8):   # sums from 3.6e38 up, no two alike, not in the groups' order
        big[g * size + 3] = 1.8e38 + 1e36 * g
        big[g * size + 5] = 1.8e38 + 1e37 * ((5 * g + 3) % 8)
    for kept in (1, 3):
        check(M, logits(30, E, 1), big, k, groups=8, kept=kept)
        check(M, logits(30, E, 2), big, k, "softmax", groups=8, kept=kept)
    check(M, logits(30, E, 3), -big, k, groups=8, kept=3)
    low = np.full(E, -np.inf, np.float32)   # groups 0 to 2: nothing at all; 3 to 7: two experts and more, hardly
    low[3 * size:] = -rng.permutation(np.linspace(3e38, 3.4e38, E - 3 * size)).astype(np.float32)
    check(M, logits(30, E, 4), low, k, groups=8, kept=2, renorm=False)


@pytest.mark.parametrize("E, k, groups, kept", [
    (8, 4, 1, 1), (8, 8, 1, 1), (16, 6, 1, 1), (32, 8, 1, 1), (64, 8, 8, 3), (64, 6, 8, 2), (48, 8, 8, 4), (48, 8, 4, 2), (128, 8, 8, 2),
    (128, 32, 1, 1), (256, 16, 1, 1), (256, 16, 8, 2), (256, 9, 4, 1), (60, 60, 1, 1), (512, 64, 1, 1), (512, 40, 32, 5), (1024, 64, 1, 1),
    (1024, 64, 64, 4), (333, 50, 3, 1),
])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_choices_of_few_lanes_and_of_many_candidates(M, score, E, k, groups, kept):
    """k near the number of lanes with an expert, or beyond it; logits that only bf16 tells apart, so that lanes
    tie; and more equal values than are ranked."""
    rng = np.random.default_rng(E + k)
    lg = logits(70, E, E * k)
    bias = (rng.standard_normal(E) * 0.1).astype(np.float32)
    check(M, lg, bias, k, score, groups, kept)
    check(M, lg, None, k, score, groups, kept, 1)
    coarse = np.round(lg * 8) / 8
    coarse[coarse == 0] = -0.0
    check(M, coarse, None, k, score, groups, kept, 1, bwd=False)
    check(M, coarse, np.zeros(E, np.float32), k, score, groups, kept, bwd=False)
    out = bias.copy()   # experts out of service, among them whole lanes
    out[rng.random(E) < 0.3] = -np.inf
    out[:4] = -np.inf
    check(M, lg, out, k, score, groups, kept, bwd=False)
    check(M, -np.exp(lg * 20).clip(1e-30, 1e30), None, k, "sigmoid", groups, kept, 1, False, bwd=False)   # over all of fp32


def microseconds(f, n=5):
    f()
    torch.cuda.synchronize()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    best = float("inf")
    for _ in range(3):
        a.record()
        for _ in range(n):
            f()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b) * 1e3 / n)
    return best


@pytest.mark.parametrize("size, beside", [
    ((8, 4, 1, 1), (8, 2, 1, 1)), ((16, 6, 1, 1), (16, 4, 1, 1)), ((64, 8, 8, 3), (64, 8, 8, 4)), ((48, 8, 4, 2), (64, 8, 8, 4)),
    ((256, 16, 1, 1), (256, 8, 1, 1)),
])
def test_no_size_leaves_the_fp32_form(M, size, beside):
    """Times at 65536 tokens, beside those of a size with more lanes than choices: one token after another in 64
    bits takes 4 to 11 times as long, the fp32 form at most about twice (k to the second at most: 16 against 8)."""
    def us(E, k, groups, kept):
        c = Call(M, logits(65536, E), np.linspace(-.1, .1, E).astype(np.float32), k, groups=groups, kept=kept)
        return microseconds(c.run)

    assert us(*size) <= 3 * us(*beside)
