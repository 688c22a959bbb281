"""The router with scores at the ends of fp32's range (GPU), against the fp64
oracle; tolerances as in test_gpu_routing.py."""
import numpy as np
import pytest

from .test_gpu_routing import M, check  # noqa: F401

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
