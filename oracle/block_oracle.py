"""fp64 oracle of the operators around a MoE block: the router with scores, bias and groups and its
gradient, 4-bit blocks, the experts' product with 4-bit weights, and the norms with their gradients. Plain
numpy, written from the formulas, one token, block or expert at a time.
"""
from __future__ import annotations

import numpy as np

from .dense_oracle import act_forward
from .moe_oracle import sigmoid

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


# ---------------------------------------------------------------- routing
def scores(row, score):
    """Scores of one token's logits; a non-finite logit scores 0 and has no part in the softmax."""
    fin = np.isfinite(row)
    s = np.zeros(len(row))
    if not fin.any():
        return s
    s[fin] = sigmoid(row[fin]) if score == "sigmoid" else np.exp(row[fin] - row[fin].max())
    return s if score == "sigmoid" else s / s.sum()


def choose(row, bias, score, k, groups=1, topk_groups=1, group_top=2):
    """The k experts of one token, best first."""
    row = np.asarray(row, dtype=np.float64)
    E = len(row)
    b = np.zeros(E) if bias is None else np.asarray(bias, dtype=np.float64)
    ok = np.isfinite(row) & np.isfinite(b)
    s = scores(row, score)
    c = np.where(ok, s + np.where(ok, b, 0.0), -np.inf)
    by = np.where(ok, row, -np.inf) if bias is None else c
    size = E // groups
    worth = []
    for g in range(groups):
        v = np.sort((c if group_top == 2 else by)[g * size:(g + 1) * size])[::-1]
        worth.append(v[0] + (v[1] if group_top == 2 and size > 1 and np.isfinite(v[1]) else 0.0))
    kept = sorted(range(groups), key=lambda g: (-worth[g], g))[:topk_groups]
    members = [e for e in range(E) if e // size in kept]
    return sorted(members, key=lambda e: (-by[e], e))[:k]


def weights(row, bias, idx, score, renorm, scale):
    """Weights of the chosen experts idx of one token."""
    row = np.asarray(row, dtype=np.float64)
    b = np.zeros(len(row)) if bias is None else np.asarray(bias, dtype=np.float64)
    idx = np.asarray(idx)
    ok = (np.isfinite(row) & np.isfinite(b))[idx]
    if renorm:   # shifted, so that scores that underflow keep their ratios
        w = np.zeros(len(idx))
        if ok.any():
            v = row[idx][ok]
            lp = -np.logaddexp(0.0, -v) if score == "sigmoid" else v
            p = np.exp(lp - lp.max())
            w[ok] = p / p.sum()
    else:
        w = np.where(ok, scores(row, score)[idx], 0.0)
    return scale * w


def route_scores(logits, bias, score, k, groups=1, topk_groups=1, group_top=2, renorm=False, scale=1.0):
    lg = np.asarray(logits, dtype=np.float64)
    idx = np.array([choose(r, bias, score, k, groups, topk_groups, group_top) for r in lg], dtype=np.int32)
    w = np.array([weights(r, bias, i, score, renorm, scale) for r, i in zip(lg, idx)])
    return idx, w


def route_scores_bwd(logits, bias, idx, ds, score, renorm=False, scale=1.0):
    """dlogits of sum(ds * w) for the given choice, through the Jacobian of every token's weights."""
    lg = np.asarray(logits, dtype=np.float64)
    b = np.zeros(lg.shape[1]) if bias is None else np.asarray(bias, dtype=np.float64)
    out = np.zeros_like(lg)
    for t, (row, ii) in enumerate(zip(lg, idx)):
        ii = np.asarray(ii)
        ok = (np.isfinite(row) & np.isfinite(b))[ii]
        s = scores(row, score)
        E = len(row)
        # d s_e / d l_f
        J = np.diag(s * (1 - s)) if score == "sigmoid" else np.diag(s) - np.outer(s, s)
        Jc = J[ii] * ok[:, None]              # [k, E]
        if renorm:
            w = weights(row, bias, ii, score, True, 1.0)
            live = np.isfinite(row)[ii]
            # d log s_j / d l_f
            L = np.zeros((len(ii), E))
            for j, e in enumerate(ii):
                if ok[j] and live[j]:
                    L[j, e] += (1 - s[e]) if score == "sigmoid" else 1.0
            g = np.asarray(ds[t], dtype=np.float64)
            out[t] = scale * ((w * (g - (w * g).sum()))[:, None] * L).sum(0)
        else:
            out[t] = scale * np.asarray(ds[t], dtype=np.float64) @ Jc
    return out


# ---------------------------------------------------------------- 4-bit blocks
def quant_mxfp4(v):
    """(codes one a value, E8M0 codes) of row-wise 32-blocks of v [R, C] (bf16 values)."""
    v = np.asarray(v, dtype=np.float64)
    R, C = v.shape
    q, s = np.zeros((R, C), np.uint8), np.zeros((R, C // 32), np.uint8)
    for r in range(R):
        for b in range(C // 32):
            x = v[r, 32 * b:32 * b + 32]
            if not np.isfinite(x).all():
                s[r, b] = 255
                continue
            amax = np.abs(x).max()
            e = -127
            if amax > 0:
                e = max(-127, int(np.floor(np.log2(amax))) - 3)
                while amax > 6.0 * 2.0**e:
                    e += 1
            y = np.abs(x) / 2.0**e
            d = np.abs(y[:, None] - E2M1[None, :])
            best = d.min(1, keepdims=True)
            # the nearer code, of two as near the even one
            code = np.array([min(np.flatnonzero(dd == bb), key=lambda c: c % 2) for dd, bb in zip(d, best[:, 0])])
            q[r, 32 * b:32 * b + 32] = code + 8 * np.signbit(x)
            s[r, b] = e + 127
    return q, s


def pack4(q):
    return (q[..., 0::2] | (q[..., 1::2] << 4)).astype(np.uint8)


def dequant_mxfp4(packed, s):
    packed = np.asarray(packed)
    q = np.empty(packed.shape[:-1] + (2 * packed.shape[-1],), np.uint8)
    q[..., 0::2], q[..., 1::2] = packed & 15, packed >> 4
    v = E2M1[q & 7] * np.where(q & 8, -1.0, 1.0)
    s = np.asarray(s).astype(np.float64)
    f = np.where(s == 255, np.nan, 2.0 ** (s - 127))
    return v * np.repeat(f, 32, axis=-1)


def grouped_linear(x, w, offsets, counts, act="none"):
    """y [rows, NO] for the experts' rows of x [rows, K], w [E, N, K]; NaN where no row is."""
    x = np.asarray(x, dtype=np.float64)
    y = None
    for e in range(len(counts)):
        a, n = int(offsets[e]), int(counts[e])
        z = act_forward(x[a:a + n] @ np.asarray(w[e], dtype=np.float64).T, act)
        if y is None:
            y = np.full((len(x), z.shape[1]), np.nan)
        y[a:a + n] = z
    return y


# ---------------------------------------------------------------- norms
def norm(x, w, eps):
    """(y, rstd)."""
    x = np.asarray(x, dtype=np.float64)
    r = 1 / np.sqrt((x * x).mean(1) + eps)
    return x * r[:, None] * np.asarray(w, dtype=np.float64), r


def norm_bwd(dy, x, w, eps):
    """(dx, dw) of norm."""
    dy, x, w = (np.asarray(v, dtype=np.float64) for v in (dy, x, w))
    r = 1 / np.sqrt((x * x).mean(1, keepdims=True) + eps)
    h, g = x * r, dy * w
    return r * (g - h * (g * h).mean(1, keepdims=True)), (dy * h).sum(0)


def _gate(gate, sig):
    if gate is None:
        return 1.0, 0.0
    g = np.asarray(gate, dtype=np.float64)
    return (sigmoid(g), sigmoid(g) * sigmoid(-g)) if sig else (g, np.ones_like(g))


def post_norm(y, x, w, eps, gate=None, sig=False, scale=1.0):
    """(out, rstd) with gate [T, 1] or [T, d]."""
    v, r = norm(y, w, eps)
    return np.asarray(x, dtype=np.float64) + scale * _gate(gate, sig)[0] * v, r


def post_norm_bwd(dout, y, w, eps, gate=None, sig=False, scale=1.0):
    """(dy, dgate or None, dw)."""
    g, slope = _gate(gate, sig)
    db = scale * np.asarray(dout, dtype=np.float64)
    dgate = None
    if gate is not None:
        full = db * norm(y, w, eps)[0]
        dgate = (full.sum(1, keepdims=True) if np.shape(gate)[1] == 1 else full) * slope
    dy, dw = norm_bwd(db * g, y, w, eps)
    return dy, dgate, dw
