"""The oracle of the operators around a MoE block: choices by brute force and by hand, gradients against
differences, 4-bit blocks exhaustively (CPU)."""
import itertools

import numpy as np
import pytest

from oracle import block_oracle as B
from oracle import moe_oracle as O


def test_choice_by_hand():
    row = np.array([0.0, 3.0, 2.0, 1.0, -1.0, 2.5])
    assert B.choose(row, None, "sigmoid", 3) == [1, 5, 2]
    # a bias moves the choice, not the weight
    bias = np.array([1.0, 0, 0, 0, 0, 0])
    assert B.choose(row, bias, "sigmoid", 2) == [0, 1]
    w = B.weights(row, bias, [0, 1], "sigmoid", False, 2.0)
    np.testing.assert_allclose(w, [1.0, 2 / (1 + np.exp(-3.0))])
    # groups (0, 1), (2, 3), (4, 5): worth by their best 3, 2, 2.5; by the sum of scores the middle one beats the last
    assert B.choose(row, None, "sigmoid", 2, 3, 2, 1) == [1, 5]
    s = 1 / (1 + np.exp(-row))
    assert s[2] + s[3] > s[4] + s[5] and s[2] + s[3] > s[0] + s[1]
    assert B.choose(row, None, "sigmoid", 2, 3, 1, 2) == [2, 3]
    # ties to the lower index; an expert out of service last, and weighing nothing
    assert B.choose(np.ones(4), None, "softmax", 3) == [0, 1, 2]
    off = np.array([-np.inf, 0, 0, -np.inf])
    assert B.choose(np.ones(4), off, "softmax", 3) == [1, 2, 0]
    np.testing.assert_allclose(B.weights(np.ones(4), off, [1, 2, 0], "softmax", True, 1.0), [0.5, 0.5, 0.0])


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [False, True])
def test_gradient_against_differences(score, renorm):
    rng = np.random.default_rng(3)
    lg, bias, ds = rng.standard_normal((5, 9)), rng.standard_normal(9) * 0.1, rng.standard_normal((5, 3))
    lg[2, 4] = np.inf
    bias[7] = -np.inf
    idx, _ = B.route_scores(lg, bias, score, 3)
    idx[1] = [2, 7, 5]     # one out of service among the chosen
    got = B.route_scores_bwd(lg, bias, idx, ds, score, renorm, 1.7)
    loss = lambda l: sum((ds[t] * B.weights(l[t], bias, idx[t], score, renorm, 1.7)).sum() for t in range(5))  # noqa: E731
    for t, e in itertools.product(range(5), range(9)):
        if not np.isfinite(lg[t, e]):
            assert got[t, e] == 0
            continue
        hi, lo = lg.copy(), lg.copy()
        hi[t, e] += 1e-5
        lo[t, e] -= 1e-5
        assert abs((loss(hi) - loss(lo)) / 2e-5 - got[t, e]) < 1e-8, (t, e)


def test_4_bit_codes_of_every_border():
    """Every code, the borders between neighbours (to the even one) and values beside them, under scale 1
    (the block's largest is 6)."""
    mids = (B.E2M1[1:] + B.E2M1[:-1]) / 2
    v = np.concatenate([B.E2M1, mids, mids * (1 - 2.0**-7), mids * (1 + 2.0**-7)])
    v = np.concatenate([v, -v, np.zeros(64 - 2 * len(v) % 64)])
    v = np.concatenate([v, np.zeros(-len(v) % 31)]).reshape(-1, 31)
    v = np.concatenate([v, np.full((len(v), 1), 6.0)], 1)
    q, s = B.quant_mxfp4(v)
    assert (s == 127).all()
    back = B.dequant_mxfp4(B.pack4(q), s)
    for x, y in zip(v.ravel(), back.ravel()):
        d = np.abs(np.abs(x) - B.E2M1)
        near = np.flatnonzero(d == d.min())
        want = B.E2M1[near[0]] if len(near) == 1 else B.E2M1[[c for c in near if c % 2 == 0][0]]
        assert abs(y) == want


def test_4_bit_scales():
    for amax, e in [(6.0, 0), (6.0625, 1), (12.0, 1), (4.0, 0), (3.0, -1), (1.0, -2), (2.0**-126, -127), (0.0, -127),
                    (2.0**127, 125), (1.9921875 * 2.0**127, 126)]:
        v = np.zeros((1, 32))
        v[0, 5] = -amax
        q, s = B.quant_mxfp4(v)
        assert s[0, 0] == e + 127, amax
    for bad in (np.nan, np.inf, -np.inf):
        v[0, 3] = bad
        q, s = B.quant_mxfp4(v)
        assert s[0, 0] == 255 and np.isnan(B.dequant_mxfp4(B.pack4(q), s)).all()


def test_norm_gradients_against_differences():
    rng = np.random.default_rng(5)
    y, x, w, do = (rng.standard_normal(s) for s in ((3, 8), (3, 8), (8,), (3, 8)))
    for cols, sig in ((0, False), (1, True), (8, True), (8, False)):
        gate = rng.standard_normal((3, cols)) if cols else None
        f = lambda y_, w_, g_: (B.post_norm(y_, x, w_, 1e-3, g_, sig, 0.7)[0] * do).sum()  # noqa: E731
        dy, dg, dw = B.post_norm_bwd(do, y, w, 1e-3, gate, sig, 0.7)
        for arr, grad, k in ((y, dy, 0), (w, dw, 1), (gate, dg, 2)):
            if arr is None:
                continue
            for i in np.ndindex(*arr.shape):
                args = [[y, w, gate], [y, w, gate]]
                for sgn, a in zip((1, -1), args):
                    a[k] = a[k].copy()
                    a[k][i] += sgn * 1e-5
                assert abs((f(*args[0]) - f(*args[1])) / 2e-5 - grad[i]) < 1e-7, (cols, k, i)


def test_product_is_the_matrix_product_of_the_values():
    rng = np.random.default_rng(9)
    x, w = rng.standard_normal((6, 64)), rng.standard_normal((2, 16, 64))
    y = B.grouped_linear(x, w, [0, 4, 6], [3, 1])
    np.testing.assert_allclose(y[:3], x[:3] @ w[0].T)
    np.testing.assert_allclose(y[4], x[4] @ w[1].T)
    assert np.isnan(y[3]).all() and np.isnan(y[5]).all()
    assert O.sigmoid(0.0) == 0.5
