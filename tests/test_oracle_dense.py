"""Pins of the dense oracle: gradients against differences, losses against closed forms (CPU)."""
import numpy as np
import pytest

from oracle import dense_oracle as D


@pytest.mark.parametrize("act", D.ACTS)
def test_linear_gradients_against_differences(act):
    rng = np.random.default_rng(3)
    T, K, N = 3, 5, 64
    x, w, b = rng.standard_normal((T, K)), rng.standard_normal((K, N)), rng.standard_normal(N)
    y, z = D.linear(x, w, act, b)
    dy = rng.standard_normal(y.shape)
    dz = D.act_backward(dy, z, act)
    loss = lambda x, w, b: (D.linear(x, w, act, b)[0] * dy).sum()  # noqa: E731
    h = 1e-5
    for grad, at, vary in ((dz @ w.T, (1, 2), lambda d: (x + d, w, b)), (x.T @ dz, (4, 37), lambda d: (x, w + d, b)),
                           (dz.sum(0), (40,), lambda d: (x, w, b + d))):
        d = np.zeros(grad.shape)
        d[at] = h
        diff = (loss(*vary(d)) - loss(*vary(-d))) / (2 * h)
        assert abs(diff - grad[at]) <= 1e-6 * (1 + abs(diff))


def test_balanced_routing_has_loss_one_and_collapse_has_loss_E():
    T, E = 16, 8
    even = np.arange(T)[:, None] % E
    r = D.balance_loss(np.zeros((T, E)), even, z_coef=0.0)
    assert np.isclose(r["loss"][1], 1.0) and np.isclose(r["loss"][2], np.log(E) ** 2)
    assert np.allclose(r["dlogits"], 0.0)
    lg = np.zeros((T, E))
    lg[:, 3] = 60.0
    r = D.balance_loss(lg, np.full((T, 1), 3))
    assert np.isclose(r["loss"][1], E)


def test_balance_gradient_against_differences():
    rng = np.random.default_rng(4)
    T, E, k = 23, 5, 2
    lg = rng.standard_normal((T, E))
    lg[7, 2] = -np.inf
    lg[9] = -np.inf
    idx = np.argsort(-lg, 1)[:, :k]
    valid = rng.random(T) < 0.7
    offs = [2, 2, 9, 20]
    run = lambda v: D.balance_loss(v, idx, valid, offs, 0.3, 0.2)  # noqa: E731
    r = run(lg)
    assert r["tokens"][-1] == r["tokens"][:-2].sum() == (valid[2:20] & np.isfinite(lg[2:20]).any(1)).sum()
    assert (r["dlogits"][~valid] == 0).all() and (r["dlogits"][:2] == 0).all() and (r["dlogits"][20:] == 0).all()
    for t in range(T):
        for e in range(E):
            if not np.isfinite(lg[t, e]):
                assert r["dlogits"][t, e] == 0
                continue
            d = np.zeros((T, E))
            d[t, e] = 1e-5
            diff = (run(lg + d)["loss"][0] - run(lg - d)["loss"][0]) / 2e-5
            assert abs(diff - r["dlogits"][t, e]) < 1e-8
