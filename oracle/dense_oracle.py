"""fp64 oracle of the dense half of the layer: the linear layer with its
activation, the backward pass, and the router losses. Plain numpy, written from
the formulas; shares the activations and the interleave of moe_oracle only.
"""
from __future__ import annotations

import numpy as np

from .moe_oracle import deinterleave, gelu, gelu_grad, interleave, sigmoid, silu

GATED = ("swiglu", "geglu")
ACTS = ("swiglu", "geglu", "srelu", "none", "silu", "gelu")  # index: the library's code


def _f(v, act):
    if act in ("silu", "swiglu"):
        return silu(v)
    if act in ("gelu", "geglu"):
        return gelu(v)
    if act == "srelu":
        return np.maximum(v, 0.0) ** 2
    return v


def _df(v, act):
    if act in ("silu", "swiglu"):
        s = sigmoid(v)
        return s * (1 + v * (1 - s))
    if act in ("gelu", "geglu"):
        return gelu_grad(v)
    if act == "srelu":
        return 2 * np.maximum(v, 0.0)
    return np.ones_like(v)


def act_forward(z, act):
    """f(z): [T, N] -> [T, N], or [T, N / 2] for a gated activation over interleaved columns."""
    z = np.asarray(z, dtype=np.float64)
    if act in GATED:
        g, u = deinterleave(z)
        return _f(g, act) * u
    return _f(z, act)


def act_backward(dy, z, act):
    """dL/dz from dL/df(z)."""
    dy, z = np.asarray(dy, dtype=np.float64), np.asarray(z, dtype=np.float64)
    if act in GATED:
        g, u = deinterleave(z)
        return interleave(dy * u * _df(g, act), dy * _f(g, act))
    return dy * _df(z, act)


def linear(x, w, act="none", bias=None, residual=None):
    """(y, z): z = x w + bias, y = f(z) + residual."""
    z = np.asarray(x, dtype=np.float64) @ np.asarray(w, dtype=np.float64)
    if bias is not None:
        z = z + np.asarray(bias, dtype=np.float64)
    y = act_forward(z, act)
    return (y if residual is None else y + np.asarray(residual, dtype=np.float64)), z


def balance_loss(logits, topk_idx, valid=None, seq_offsets=None, balance_coef=1.0, z_coef=1.0):
    """dict of loss [total, balance, z], counts [S, E], prob [S, E], tokens [S + 2] and dlogits
    [T, E] (the gradient of the total), as include/moe.h defines them. One token at a time."""
    lg = np.asarray(logits, dtype=np.float64)
    idx = np.asarray(topk_idx)
    T, E = lg.shape
    k = idx.shape[1]
    offs = np.array([0, T]) if seq_offsets is None else np.asarray(seq_offsets)
    S = len(offs) - 1
    fin = np.isfinite(lg)
    live = fin.any(1) & (np.ones(T, bool) if valid is None else np.asarray(valid) != 0)
    seq = np.full(T, -1)
    for s in range(S):
        seq[offs[s]:offs[s + 1]] = s
    live &= seq >= 0
    p = np.zeros((T, E))
    lse = np.zeros(T)
    counts = np.zeros((S, E), dtype=np.int64)
    psum = np.zeros((S, E))
    n = np.zeros(S, dtype=np.int64)
    for t in np.flatnonzero(live):
        top = lg[t][fin[t]].max()
        e = np.where(fin[t], np.exp(np.where(fin[t], lg[t], top) - top), 0.0)
        p[t] = e / e.sum()
        lse[t] = top + np.log(e.sum())
        s = seq[t]
        n[s] += 1
        psum[s] += p[t]
        for j in range(k):
            if 0 <= idx[t, j] < E:
                counts[s, idx[t, j]] += 1
    some = n > 0
    per = np.maximum(n, 1)[:, None]
    prob, f = psum / per, counts * E / (k * per)
    nlive, ntot = int(some.sum()), int(n.sum())
    bal = (f * prob).sum() / max(nlive, 1)
    z = (lse ** 2).sum() / max(ntot, 1)
    d = np.zeros((T, E))
    for t in np.flatnonzero(live):
        s = seq[t]
        d[t] = balance_coef / (nlive * n[s]) * p[t] * (f[s] - (f[s] * p[t]).sum())
        d[t] += z_coef * 2 * lse[t] / ntot * p[t]
    return {"loss": np.array([balance_coef * bal + z_coef * z, bal, z]), "counts": counts, "prob": prob,
            "tokens": np.concatenate([n, [nlive, ntot]]), "dlogits": d}
