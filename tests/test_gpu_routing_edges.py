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
