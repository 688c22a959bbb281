"""The router where a workgroup takes several passes of tokens (more than 16384 of them with 16 lanes a token, 4096
with 64): every choice, weight, row and gradient, against the formulas in 64 bits (GPU). Tolerances as in
test_gpu_routing.py."""
import numpy as np
import pytest
import torch

from oracle import block_oracle as B
from oracle import moe_oracle as O

from ._util import f32_tensor
from .test_gpu_routing import M, TOL, Call, logits  # noqa: F401

pytestmark = pytest.mark.gpu


def reference(lg, bias, score, k, groups, kept, top, renorm, scale, ds):
    """(idx, w, dlogits), all tokens at once; finite logits, biases finite or -inf, k available experts a token."""
    x = lg.astype(np.float64)
    T, E = x.shape
    if score == "sigmoid":
        s = 1 / (1 + np.exp(-x))
    else:
        s = np.exp(x - x.max(1, keepdims=True))
        s /= s.sum(1, keepdims=True)
    by = x if bias is None else s + bias.astype(np.float64)
    if groups > 1:
        c = s if bias is None and top == 2 else by
        best = -np.sort(-c.reshape(T, groups, -1), 2)[:, :, :top]
        worth = np.where(np.isfinite(best) | (np.arange(best.shape[2]) == 0), best, 0.0).sum(2)
        order = np.argsort(-worth, 1, kind="stable")[:, :kept]
        keep = np.zeros((T, groups), bool)
        np.put_along_axis(keep, order, True, 1)
        by = np.where(np.repeat(keep, E // groups, 1), by, -np.inf)
    idx = np.argsort(-by, 1, kind="stable")[:, :k]
    assert np.isfinite(np.take_along_axis(by, idx, 1)).all()
    p, v = np.take_along_axis(s, idx, 1), np.take_along_axis(x, idx, 1)
    slope = 1 / (1 + np.exp(v)) if score == "sigmoid" else np.ones_like(v)
    d = np.zeros_like(x)
    if renorm:
        w = p / p.sum(1, keepdims=True)
        np.put_along_axis(d, idx, scale * w * slope * (ds - (w * ds).sum(1, keepdims=True)), 1)
    else:
        w = p
        np.put_along_axis(d, idx, scale * p * slope * ds, 1)
        if score == "softmax":
            d -= scale * s * (p * ds).sum(1, keepdims=True)
    return idx, scale * w, d


def test_reference_is_the_oracles():
    lg, ds = logits(9, 24, 3), np.random.default_rng(2).standard_normal((9, 4))
    bias = np.linspace(-.2, .2, 24).astype(np.float32)
    bias[5] = -np.inf
    for score in ("sigmoid", "softmax"):
        for b in (None, bias):
            for top, renorm in ((1, False), (2, True), (2, False)):
                idx, w, d = reference(lg, b, score, 4, 6, 3, top, renorm, 1.5, ds)
                i, v = B.route_scores(lg, b, score, 4, 6, 3, top, renorm, 1.5)
                assert np.array_equal(idx, i)
                np.testing.assert_allclose(w, v, rtol=1e-12)
                np.testing.assert_allclose(d, B.route_scores_bwd(lg, b, i, ds, score, renorm, 1.5), rtol=1e-9, atol=1e-14)


@pytest.mark.parametrize("T, E, k, score, bias, groups, kept, top, renorm", [
    (20001, 256, 8, "sigmoid", True, 8, 4, 2, True),    # 16 lanes a token, rows in 16-byte pieces
    (33000, 256, 8, "softmax", True, 8, 3, 1, False),   # three passes
    (17000, 128, 16, "sigmoid", False, 4, 2, 2, True),
    (18000, 54, 6, "sigmoid", True, 9, 4, 2, False),    # rows that go through LDS
    (16500, 102, 5, "softmax", False, 6, 2, 1, True),
    (40000, 8, 4, "sigmoid", True, 1, 1, 2, True),      # fewer lanes with an expert than choices
    (5001, 512, 8, "sigmoid", True, 16, 4, 2, True),    # 64 lanes a token
    (9000, 200, 20, "softmax", True, 5, 3, 2, False),
    (4500, 1023, 9, "sigmoid", True, 3, 2, 2, True),
    (4200, 333, 40, "softmax", False, 1, 1, 1, False),
])
def test_several_passes_of_tokens(M, T, E, k, score, bias, groups, kept, top, renorm):
    lg = logits(T, E, T)
    rng = np.random.default_rng(E)
    b = (rng.standard_normal(E) * 0.1).astype(np.float32) if bias else None
    if bias and E > 8:
        b[rng.integers(E)] = -np.inf
    ds = rng.standard_normal((T, k)).astype(np.float32)
    idx, w, d = reference(lg, b, score, k, groups, kept, top, renorm, 1.5, ds.astype(np.float64))
    c = Call(M, lg, b, k, score, groups, kept, top, renorm, 1.5).run()
    got = c.idx.cpu().numpy()
    assert np.array_equal(got, idx), np.flatnonzero((got != idx).any(1))[:5]
    for name, want in zip(("counts", "offsets", "row_of", "src_of"), O.layout(idx, E, c.cap)):
        assert np.array_equal(getattr(c, name).cpu().numpy(), want), name
    np.testing.assert_allclose(c.w.cpu().numpy(), w, rtol=TOL)
    assert int(c.err) == 0
    most = np.abs(w).max(1, keepdims=True) * np.abs(ds).max(1, keepdims=True)
    assert (np.abs(c.bwd(f32_tensor(ds)).dlogits.cpu().numpy() - d) <= 2 * TOL * most).all()


@pytest.mark.parametrize("T, E, k", [(20000, 64, 8), (6000, 512, 24)])
def test_tokens_in_doubt_in_every_pass(M, T, E, k):
    """Biases that make up for the scores to a part in 2^30, for every third token: it is chosen in 64 bits, between
    others that are not."""
    rng = np.random.default_rng(T)
    row = logits(1, E, 1)[0]
    lg = np.where((np.arange(T) % 3 == 0)[:, None], row, logits(T, E, 2)).astype(np.float32)
    bias = (0.75 - 1 / (1 + np.exp(-row.astype(np.float64))) + rng.integers(-3, 4, E) * 2.0**-30).astype(np.float32)
    idx, w, _ = reference(lg, bias, "sigmoid", k, 8, 4, 2, True, 1.0, np.zeros((T, k)))
    c = Call(M, lg, bias, k, groups=8, kept=4).run()
    assert np.array_equal(c.idx.cpu().numpy(), idx)
    np.testing.assert_allclose(c.w.cpu().numpy(), w, rtol=TOL)
    assert torch.equal(c.counts.cpu(), torch.from_numpy(np.bincount(idx.ravel(), minlength=E)).int())
