"""Cases of what surrounds and fills a mixture-of-experts block: the router that
scores experts with a balance bias, in groups, and its gradient; 4-bit block
quantisation and the experts' products with 4-bit weights; and the norms before
and after the block, the latter fused with the experts' combination, a gate and
the scaled residual, with their gradients.

A 4-bit block is 32 neighbouring values: E2M1 codes (0, .5, 1, 1.5, 2, 3, 4, 6
and their negatives, two codes a byte, the first in the low half) and one E8M0
scale, the smallest power of two that keeps the block's largest magnitude within
6. An 8-bit block holds E4M3 codes (within 448). Expert weights are [E, N, K],
blocks along K; a gated layer's N has 32 gate and 32 up channels in turn. Rows
of the experts' buffer: expert e owns counts[e] rows from offsets[e], a multiple
of 128, in the order of the (token, choice) pairs.
"""
import math

import torch

own = False

GATED = ("swiglu", "geglu")
EPS = 1e-6


def listed():
    return [
        # a decode step of 16 sequences, sigmoid scores, balance bias, 4 of 8 groups: latency
        {"name": "route-decode", "op": "route", "T": 16, "E": 256, "k": 8, "score": "sigmoid", "bias": True, "dead": 0,
         "groups": 8, "kept": 4, "top": 2, "renorm": True, "scale": 2.5, "bwd": False},
        # a ragged micro-batch, softmax scores, groups by their best expert, with the gradient
        {"name": "route-odd", "op": "route", "T": 1021, "E": 160, "k": 6, "score": "softmax", "bias": False, "dead": 0,
         "groups": 8, "kept": 3, "top": 1, "renorm": False, "scale": 16.0, "bwd": True},
        # a training step's tokens, sigmoid scores, balance bias, groups, with the gradient
        {"name": "route-train", "op": "route", "T": 131072, "E": 256, "k": 8, "score": "sigmoid", "bias": True, "dead": 0,
         "groups": 8, "kept": 4, "top": 2, "renorm": True, "scale": 2.5, "bwd": True},
        # a ragged prompt's tokens to 4 bits, on the way into a product
        {"name": "quant-tokens", "op": "quant", "B": 1, "R": 1021, "C": 2880, "col": False},
        # a layer's gate/up weights [d, 2n] to 4 bits along d, as a server lays them out
        {"name": "quant-weights", "op": "quant", "B": 8, "R": 7168, "C": 4096, "col": True},
        # one token through its 8 experts' gate/up projection, bf16 activations: the read of the weights
        {"name": "experts-one-token", "op": "experts", "T": 1, "k": 8, "E": 32, "K": 7168, "N": 4096, "act": "swiglu", "x": "bf16", "gather": True},
        # a ragged prompt through a down projection from 8-bit activations
        {"name": "experts-prompt", "op": "experts", "T": 1021, "k": 8, "E": 32, "K": 2048, "N": 7168, "act": "none", "x": "mxfp8", "gather": False},
        # prefill through the gate/up projection from 4-bit activations
        {"name": "experts-prefill", "op": "experts", "T": 16384, "k": 8, "E": 32, "K": 7168, "N": 4096, "act": "swiglu", "x": "mxfp4", "gather": True},
        # the norm before a block in a decode step, with the residual sum
        {"name": "norm-decode", "op": "norm", "T": 8, "d": 7168, "res": True, "bwd": False},
        # the same of a training step, with the gradient
        {"name": "norm-train", "op": "norm", "T": 32768, "d": 8192, "res": True, "bwd": True},
        # after the block, a ragged micro-batch of a 2880-wide model, one gate a token
        {"name": "post-odd", "op": "post", "T": 1021, "d": 2880, "k": 4, "E": 32, "gate": "token", "sigmoid": True, "scale": 1.0, "bwd": True},
        # after the block, a training step: 8 experts combined, a gate a channel, scaled residual branch
        {"name": "post-train", "op": "post", "T": 16384, "d": 7168, "k": 8, "E": 32, "gate": "full", "sigmoid": True, "scale": 0.5, "bwd": True},
    ]


def _log(rng, lo, hi, step=1):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(lo, min(hi, v // step * step))


def draw(rng):
    op = rng.choice(["route", "route", "quant", "experts", "experts", "norm", "post"])
    if op == "route":
        groups = rng.choice([1, 1, 4, 8])
        E = groups * _log(rng, 2, 256 // groups)
        kept = rng.randint(max(1, groups // 4), groups)
        score, k = rng.choice(["sigmoid", "softmax"]), rng.randint(1, min(8, kept * (E // groups)))
        return {"op": op, "T": _log(rng, 1, 131072), "E": E, "k": k, "score": score,
                "bias": rng.random() < 0.6, "dead": int(k < kept * (E // groups) and rng.random() < 0.3), "groups": groups, "kept": kept, "top": rng.randint(1, 2),
                "renorm": k > 1 and rng.random() < 0.7, "scale": rng.choice([1.0, 2.5]), "bwd": rng.random() < 0.6}  # a lone weight of 1 has no gradient
    if op == "quant":
        if rng.random() < 0.5:
            return {"op": op, "B": 1, "R": _log(rng, 1, 32768), "C": _log(rng, 32, 7168, 32), "col": False}
        return {"op": op, "B": rng.randint(1, 8), "R": _log(rng, 32, 7168, 32), "C": _log(rng, 8, 4096, 8), "col": True}
    if op == "experts":
        act = rng.choice(["swiglu", "geglu", "none", "none"])
        E = rng.choice([4, 8, 16, 32, 32])
        T, k = _log(rng, 1, 16384), rng.randint(1, min(8, E))
        K, N = _log(rng, 64, 8192, 32), _log(rng, 64, 8192, 64 if act in GATED else 8)
        N = min(N, 7168 * 4096 // K // 64 * 64)  # the weights no larger than the largest listed ones
        T = max(1, min(T, 131072 * 7168 * 4096 // (k * K * N)))
        return {"op": op, "T": T, "k": k, "E": E, "K": K, "N": N, "act": act, "x": rng.choice(["bf16", "mxfp8", "mxfp4"]),
                "gather": rng.random() < 0.5}
    if op == "norm":
        return {"op": op, "T": _log(rng, 1, 32768), "d": _log(rng, 64, 8192, 8), "res": rng.random() < 0.5, "bwd": rng.random() < 0.5}
    k = rng.choice([0, 1, 2, 4, 8])
    T, d = _log(rng, 1, 32768), _log(rng, 64, 8192, 8)
    T = min(T, 16384 * 8 * 7168 // (max(k, 1) * d))
    return {"op": op, "T": T, "d": d, "k": k, "E": 32, "gate": rng.choice(["none", "token", "full"]), "sigmoid": rng.random() < 0.5,
            "scale": rng.choice([1.0, 0.5, 0.22]), "bwd": rng.random() < 0.5}


# ---------------------------------------------------------------- block formats
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
#: between neighbouring codes: a value on the border goes to the even code
E2M1_BORDERS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)


def _block_exp(v, most):
    """Smallest e with the block's largest magnitude <= most * 2^e, within E8M0; v [..., 32] float32, most = m 2^p, m in [0.5, 1)."""
    m, p = math.frexp(most)
    f, x = torch.frexp(v.abs().amax(-1))
    e = torch.where(f > m, x - p + 1, x - p).clamp(-127, 127)
    return torch.where(f == 0, torch.full_like(e, -127), e)


def _to_mx4(v):
    """Codes (one a byte) and scales of the last dimension's blocks of a float32 tensor holding bf16 values."""
    b = v.unflatten(-1, (-1, 32))
    e = _block_exp(b, 6.0)
    a = torch.ldexp(b, -e.unsqueeze(-1))
    mag = a.abs()
    q = torch.zeros_like(mag, dtype=torch.uint8)
    for i, edge in enumerate(E2M1_BORDERS):
        q += (mag > edge) if i % 2 == 0 else (mag >= edge)
    q += 8 * torch.signbit(b)
    return q.flatten(-2), (e + 127).to(torch.uint8)


def _pack4(q):
    return q[..., 0::2] | (q[..., 1::2] << 4)


def _to_mx8(v):
    b = v.unflatten(-1, (-1, 32))
    e = _block_exp(b, 448.0)
    q = torch.ldexp(b, -e.unsqueeze(-1)).to(torch.float8_e4m3fn).view(torch.uint8)
    return q.flatten(-2), (e + 127).to(torch.uint8)


def _scale(v, s):
    return torch.ldexp(v.unflatten(-1, (-1, 32)), s.to(torch.int32).unsqueeze(-1) - 127).flatten(-2)


def _from_mx4(packed, s):
    """float32 values of packed codes [..., K / 2] and scales [..., K / 32]."""
    lut = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=packed.device)
    q = torch.stack((packed & 15, packed >> 4), -1).flatten(-2)
    return _scale(lut[q.int()], s)


def _from_mx8(q, s):
    return _scale(q.view(torch.float8_e4m3fn).float(), s)


# ---------------------------------------------------------------- inputs
def _plan(idx, E):
    """The experts' rows of the choices idx [T, k]: counts, offsets, row_of, src_of."""
    T, k = idx.shape
    flat = idx.reshape(-1).long()
    counts = torch.bincount(flat, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=idx.device)
    offsets[1:] = ((counts + 127) // 128 * 128).cumsum(0)
    order = torch.sort(flat, stable=True).indices
    first = counts.cumsum(0) - counts
    rank = torch.arange(T * k, device=idx.device) - first[flat[order]]
    row_of = torch.empty_like(flat)
    row_of[order] = offsets[flat[order]] + rank
    src_of = torch.full(((T * k + 127) // 128 * 128 + 128 * E,), -1, dtype=torch.int32, device=idx.device)
    src_of[row_of] = torch.arange(T * k, device=idx.device, dtype=torch.int32)
    return counts.int(), offsets.int(), row_of.int(), src_of


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    bf, f32, dev = torch.bfloat16, torch.float32, "cuda"

    def normal(*shape, std=1.0, mean=0.0, dtype=bf):
        return (torch.randn(*shape, device=dev, generator=g) * std + mean).to(dtype)

    st = {"case": case}
    if case["op"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        popular = torch.randperm(E, device=dev, generator=g) + 1  # a few experts are asked for more
        st["logits"] = torch.randn(T, E, device=dev, generator=g) - 0.3 * popular.log()
        st["bias"] = normal(E, std=0.05, dtype=f32) if case["bias"] else None
        if case["dead"]:  # an expert out of service
            st["bias"] = torch.zeros(E, device=dev) if st["bias"] is None else st["bias"]
            st["bias"][seed % E] = -math.inf
        st["ds"] = normal(T, k, dtype=f32)
    elif case["op"] == "quant":
        x = torch.randn(case["B"], case["R"], case["C"], device=dev, generator=g)
        x *= 1 + 20 * (torch.rand(x.shape[-1], device=dev, generator=g) < 0.01)  # a few loud channels
        st["v"] = x.to(bf)
    elif case["op"] == "experts":
        T, k, E, K, N = (case[c] for c in ("T", "k", "E", "K", "N"))
        idx = torch.randn(T, E, device=dev, generator=g).topk(k, dim=1).indices
        st["counts"], st["offsets"], st["row_of"], st["src_of"] = _plan(idx, E)
        st["plan"] = list(zip(st["offsets"].tolist(), st["counts"].tolist()))
        # weights: an expert's codes from another's by swapping halves, so that making them is quick
        w = normal(N, K, std=K**-0.5).float()
        q, s = _to_mx4(w)
        q = _pack4(q)
        st["w_q"] = torch.stack([q.roll(int(n), 0) for n in torch.randint(0, N, (E,), generator=torch.Generator().manual_seed(seed))])
        st["w_s"] = (s + torch.randint(0, 2, (E, N, K // 32), device=dev, generator=g, dtype=torch.uint8)).contiguous()
        x = normal(T, K)
        if not case["gather"]:  # the experts' buffer itself; its padding rows hold zeros
            rows = torch.zeros(len(st["src_of"]), K, dtype=bf, device=dev)
            rows[st["row_of"].long()] = x.repeat_interleave(k, 0)
            x = rows
        if case["x"] == "bf16":
            st["x"], st["x_s"] = x, None
        else:
            q, st["x_s"] = (_to_mx8 if case["x"] == "mxfp8" else _to_mx4)(x.float())
            st["x"] = q if case["x"] == "mxfp8" else _pack4(q)
    elif case["op"] == "norm":
        T, d = case["T"], case["d"]
        st["x"], st["res"] = normal(T, d), normal(T, d) if case["res"] else None
        st["w"] = normal(d, std=0.2, mean=1.0)
        st["dy"], st["dres"] = normal(T, d), normal(T, d)
    else:
        T, d, k = case["T"], case["d"], case["k"]
        st["x"], st["w"] = normal(T, d), normal(d, std=0.2, mean=1.0)
        if k:
            idx = torch.randn(T, case["E"], device=dev, generator=g).topk(k, dim=1).indices
            st["row_of"], src_of = _plan(idx, case["E"])[2:]
            st["y"] = normal(len(src_of), d, std=0.5)
            st["topk_w"] = torch.softmax(torch.randn(T, k, device=dev, generator=g), 1)
            # what the backward pass finds kept of the forward: the block's output, and the norm's statistics
            saved = (st["y"][st["row_of"].long()].reshape(T, k, d).float() * st["topk_w"].unsqueeze(2)).sum(1).to(bf)
        else:
            saved = st["y"] = normal(T, d, std=0.5)
        st["saved"], st["rstd"] = saved, torch.rsqrt(saved.float().square().mean(1) + EPS)
        st["gate"] = None if case["gate"] == "none" else normal(T, 1 if case["gate"] == "token" else d)
        st["dout"] = normal(T, d)
    return st


# ---------------------------------------------------------------- plain forms
def _chosen(st):
    """The experts of every token, best first, ties to the lower index; in 64 bits: two of them may lie close."""
    c, lg, bias = st["case"], st["logits"].double(), st["bias"]
    T, E, G = c["T"], c["E"], c["groups"]
    s = torch.sigmoid(lg) if c["score"] == "sigmoid" else torch.softmax(lg, 1)
    by = lg if bias is None else s + bias.double()  # without a bias the scores' order is the logits'
    if G > 1:
        best = (s if bias is None else by).reshape(T, G, -1).topk(min(c["top"], E // G), dim=2).values
        best = torch.where(torch.isinf(best[..., :1]), best[..., 0:1], best.where(~torch.isinf(best), 0)).sum(2)
        order = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :c["kept"]]
        keep = torch.zeros(T, G, dtype=torch.bool, device=lg.device).scatter_(1, order, True)
        keep = keep.repeat_interleave(E // G, 1)
        place = torch.where(keep, by, torch.full_like(by, -math.inf))
        # an expert of a group that was not kept comes after every one of a kept group
        first = torch.sort(keep.int(), dim=1, descending=True, stable=True).indices
        within = torch.sort(place.gather(1, first), dim=1, descending=True, stable=True).indices
        idx = first.gather(1, within)[:, :c["k"]]
    else:
        idx = torch.sort(by, dim=1, descending=True, stable=True).indices[:, :c["k"]]
    return idx, s.float()


def _route_plain(st):
    c, lg = st["case"], st["logits"]
    idx, s = _chosen(st)
    live = torch.ones_like(idx, dtype=torch.float32) if st["bias"] is None else (st["bias"][idx] > -math.inf).float()
    p = s.gather(1, idx) * live
    total = p.sum(1, keepdim=True)
    w = c["scale"] * (p / total if c["renorm"] else p)
    counts, offsets, row_of, src_of = _plan(idx, c["E"])
    out = {"idx": idx.int(), "w": w, "counts": counts, "offsets": offsets, "row_of": row_of, "src_of": src_of}
    if c["bwd"]:
        ds = st["ds"] * c["scale"]
        dp = (ds - (ds * p).sum(1, keepdim=True) / total) / total if c["renorm"] else ds
        dp = dp * live
        if c["score"] == "sigmoid":
            dl = torch.zeros_like(lg).scatter_(1, idx, dp * p * torch.sigmoid(-lg.gather(1, idx)))
        else:
            dl = torch.zeros_like(lg).scatter_(1, idx, dp * p) - s * (dp * p).sum(1, keepdim=True)
        out["dlogits"] = dl
    return out


def _act(z, act):
    h = z.reshape(z.shape[0], -1, 2, 32)
    a, u = h[:, :, 0], h[:, :, 1]
    a = a * torch.sigmoid(a) if act == "swiglu" else a * 0.5 * (1 + torch.erf(a * math.sqrt(0.5)))
    return (a * u).reshape(z.shape[0], -1)


def _experts_plain(st):
    c = st["case"]
    x = st["x"].float() if c["x"] == "bf16" else (_from_mx8 if c["x"] == "mxfp8" else _from_mx4)(st["x"], st["x_s"])
    y = torch.zeros(len(st["src_of"]), c["N"] // 2 if c["act"] in GATED else c["N"], device=x.device)
    for e, (row, n) in enumerate(st["plan"]):
        if n:
            rows = x[st["src_of"][row:row + n].long() // c["k"]] if c["gather"] else x[row:row + n]
            z = rows @ _from_mx4(st["w_q"][e], st["w_s"][e]).t()
            y[row:row + n] = _act(z, c["act"]) if c["act"] in GATED else z
    return {"y": y.to(torch.bfloat16)}


def _norm_plain(st):
    c, bf = st["case"], torch.bfloat16
    out, s = {}, st["x"].float()
    if c["res"]:
        out["total"] = (s + st["res"].float()).to(bf)  # the residual stream is bf16: the norm is of what it holds
        s = out["total"].float()
    w = st["w"].float()
    r = torch.rsqrt(s.square().mean(1, keepdim=True) + EPS)
    h = s * r
    out["y"], out["rstd"] = (h * w).to(bf), r.squeeze(1)
    if c["bwd"]:
        dy = st["dy"].float()
        g = dy * w
        out["dx"] = (r * (g - h * (g * h).mean(1, keepdim=True)) + st["dres"].float()).to(bf)
        out["dw"] = (dy * h).sum(0)
    return out


def _post_plain(st):
    c, bf = st["case"], torch.bfloat16
    out, k = {}, c["k"]
    y = st["y"].float()
    if k:
        y = (y[st["row_of"].long()].reshape(c["T"], k, -1) * st["topk_w"].unsqueeze(2)).sum(1)
        out["total"] = y.to(bf)  # the block's output is bf16: the norm is of what it holds
        y = out["total"].float()
    w = st["w"].float()
    r = torch.rsqrt(y.square().mean(1, keepdim=True) + EPS)
    h = y * r
    v = h * w
    gate = torch.ones(1, 1, device=y.device) if st["gate"] is None else st["gate"].float()
    slope = torch.ones_like(gate)
    if c["sigmoid"] and st["gate"] is not None:
        gate, slope = torch.sigmoid(gate), torch.sigmoid(gate) * torch.sigmoid(-gate)
    out["out"], out["rstd"] = (st["x"].float() + c["scale"] * gate * v).to(bf), r.squeeze(1)
    if c["bwd"]:
        db = c["scale"] * st["dout"].float()
        r = st["rstd"].unsqueeze(1)
        h = st["saved"].float() * r
        v = h * w
        if c["gate"] == "full":
            out["dgate"] = (db * v * slope).to(bf)
        elif c["gate"] == "token":
            out["dgate"] = (db * v).sum(1, keepdim=True) * slope
        dv = db * gate
        g = dv * w
        out["dy"] = (r * (g - h * (g * h).mean(1, keepdim=True))).to(bf)
        out["dw"] = (dv * h).sum(0)
    return out


def _quant_plain(st):
    v = st["v"].float()
    q, s = _to_mx4(v.transpose(1, 2).contiguous() if st["case"]["col"] else v)
    lut = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=v.device)
    return {"v": _scale(lut[q.int()], s).to(torch.bfloat16), "s": s}


def _plain(st):
    return {"route": _route_plain, "quant": _quant_plain, "experts": _experts_plain, "norm": _norm_plain, "post": _post_plain}[st["case"]["op"]](st)


# ---------------------------------------------------------------- the framework's operators
def _own(st):
    from ragged_grouped_gemm_device_amd import moe as M

    c = st["case"]
    bf, f32, i32, u8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
    b = st.get("buf")
    if b is None:  # outputs and workspace, allocated once and kept as a training or serving loop keeps them
        b = st["buf"] = {}

        def new(name, dtype, *shape):
            b[name] = torch.zeros(*shape, dtype=dtype, device="cuda")

        if c["op"] == "route":
            T, E, k = c["T"], c["E"], c["k"]
            new("idx", i32, T, k)
            new("w", f32, T, k)
            new("counts", i32, E)
            new("offsets", i32, E + 1)
            new("row_of", i32, T * k)
            new("src_of", i32, M.moe_capacity_rows(T, k, E))
            new("err", i32, 1)
            new("dlogits", f32, T, E)
            new("ws", u8, max(16, M.moe_route_scores_workspace_bytes(T, k, E)))
            b["how"] = M.Routing(score=M.MOE_SCORE_SIGMOID if c["score"] == "sigmoid" else M.MOE_SCORE_SOFTMAX, bias=st["bias"],
                                 groups=c["groups"], topk_groups=c["kept"], group_top=c["top"], renorm=c["renorm"], scale=c["scale"])
        elif c["op"] == "quant":
            B, n, K = (c["B"], c["C"], c["R"]) if c["col"] else (c["B"], c["R"], c["C"])
            new("q", u8, B, n, K // 2)
            new("s", u8, B, n, K // 32)
            new("v", bf, B, n, K)
        elif c["op"] == "experts":
            new("y", bf, len(st["src_of"]), c["N"] // 2 if c["act"] in GATED else c["N"])
            new("ws", u8, max(16, M.moe_grouped_linear_mxfp4_workspace_bytes(c["T"], c["k"], c["E"], c["K"], c["N"])))
        else:
            T, d = c["T"], c["d"]
            for name in ("total", "y", "out", "dx", "dy"):
                new(name, bf, T, d)
            new("rstd", f32, T)
            new("dw", f32, d)
            if c.get("gate") in ("token", "full"):
                new("dgate", f32 if c["gate"] == "token" else bf, *st["gate"].shape)
            new("ws", u8, max(16, M.moe_norm_workspace_bytes(T, d)))
    if c["op"] == "route":
        M.moe_route_scores(st["logits"], c["k"], b["idx"], b["w"], b["counts"], b["offsets"], b["row_of"], b["src_of"], b["err"],
                           b["ws"], b["how"])
        keys = ["idx", "w", "counts", "offsets", "row_of", "src_of"]
        if c["bwd"]:
            M.moe_route_scores_bwd(st["logits"], b["idx"], st["ds"], b["dlogits"], b["how"])
            keys.append("dlogits")
        return {key: b[key] for key in keys}
    if c["op"] == "quant":
        if c["col"]:
            M.moe_quant_mxfp4(st["v"], M.MOE_QUANT_COLWISE, q_col=b["q"], s_col=b["s"])
        else:
            M.moe_quant_mxfp4(st["v"], M.MOE_QUANT_ROWWISE, q_row=b["q"], s_row=b["s"])
        M.moe_dequant_mxfp4(b["q"].flatten(0, 1), b["s"].flatten(0, 1), b["v"].flatten(0, 1))
        return {"v": b["v"], "s": b["s"]}
    if c["op"] == "experts":
        acts = {"swiglu": M.MOE_ACT_SWIGLU, "geglu": M.MOE_ACT_GEGLU, "none": M.MOE_ACT_NONE}
        M.moe_grouped_linear_mxfp4(st["x"], st["w_q"], st["w_s"], st["offsets"], st["counts"], b["y"], c["T"], c["k"], act=acts[c["act"]],
                                   x_s=st["x_s"], src_of=st["src_of"] if c["gather"] else None, workspace=b["ws"])
        return {"y": b["y"]}
    if c["op"] == "norm":
        M.moe_norm_fwd(st["x"], st["w"], b["y"], b["rstd"], EPS, residual=st["res"], total=b["total"] if c["res"] else None)
        keys = (["total"] if c["res"] else []) + ["y", "rstd"]
        if c["bwd"]:
            M.moe_norm_bwd(st["dy"], b["total"] if c["res"] else st["x"], st["w"], b["rstd"], b["dx"], b["dw"], b["ws"], dres=st["dres"])
            keys += ["dx", "dw"]
        return {key: b[key] for key in keys}
    gate_act = M.MOE_GATE_SIGMOID if c["sigmoid"] else M.MOE_GATE_LINEAR
    rows = {"row_of": st["row_of"], "topk_w": st["topk_w"], "total": b["total"]} if c["k"] else {}
    M.moe_post_norm_fwd(st["y"], st["x"], st["w"], b["out"], b["rstd"], EPS, gate=st["gate"], gate_act=gate_act, scale=c["scale"], **rows)
    keys = (["total"] if c["k"] else []) + ["out", "rstd"]
    if c["bwd"]:
        M.moe_post_norm_bwd(st["dout"], st["saved"], st["w"], st["rstd"], b["dy"], b["dw"], b["ws"], gate=st["gate"],
                            dgate=b.get("dgate"), gate_act=gate_act, scale=c["scale"])
        keys += (["dgate"] if "dgate" in b else []) + ["dy", "dw"]
    return {key: b[key] for key in keys}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- least work
def work(case):
    op = case["op"]
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        nbytes = 4 * T * E + 8 * T * k + 4 * T * k + 4 * ((T * k + 127) // 128 * 128 + 128 * E) + (4 * E if case["bias"] else 0)
        # the gradient of a sigmoid needs the chosen logits alone, a softmax's all of them, at hand from the forward
        return {"bytes": nbytes + (4 * T * E + 4 * T * k if case["bwd"] else 0), "flops": (10 + (6 if case["bwd"] else 0)) * T * E}
    if op == "quant":
        n = case["B"] * case["R"] * case["C"]
        return {"bytes": 2 * n + 2 * n + n // 32, "flops": 0}
    if op == "experts":
        T, k, E, K, N = (case[c] for c in ("T", "k", "E", "K", "N"))
        hit = E * (1 - (1 - k / E) ** T)  # experts that some token asks for, on average
        per = {"bf16": 2.0, "mxfp8": 1 + 1 / 32, "mxfp4": 0.5 + 1 / 32}[case["x"]]
        rows = T if case["gather"] else T * k
        return {"bytes": int(hit * N * K * (0.5 + 1 / 32) + rows * K * per + 2 * T * k * (N // 2 if case["act"] in GATED else N)),
                "flops": 2 * T * k * K * N}
    T, d = case["T"], case["d"]
    if op == "norm":
        fwd = (4 if case["res"] else 2) * 2 * T * d
        return {"bytes": fwd + (3 * 2 * T * d + 6 * d if case["bwd"] else 0), "flops": (4 + (9 if case["bwd"] else 0)) * T * d}
    k = case["k"]
    gate = {"none": 0, "token": 2 * T, "full": 2 * T * d}[case["gate"]]
    # forward: the experts' rows (or their sum), x, the gate; out, and the sum where the block's rows were combined
    fwd = 2 * T * d * (max(k, 1) + 2 + (1 if k else 0)) + 8 * T * k + gate
    # backward: dout, the gate's gradient, dy; the sum and the gate are at hand from the forward
    return {"bytes": fwd + (2 * 2 * T * d + gate + 6 * d if case["bwd"] else 0), "flops": (2 * k + 6 + (14 if case["bwd"] else 0)) * T * d}


# ---------------------------------------------------------------- 64-bit values
def exact(case, seed):
    st = prepare(case, seed)
    D, op = torch.float64, case["op"]

    def e2m1(packed, s):
        """Values of 4-bit codes from their sign, exponent and fraction bits."""
        q = torch.empty(*packed.shape[:-1], 2 * packed.shape[-1], dtype=torch.int32, device=packed.device)
        q[..., 0::2], q[..., 1::2] = packed % 16, packed // 16
        ex, fr = q >> 1 & 3, (q & 1).to(D)
        v = torch.where(ex > 0, (1 + fr / 2) * torch.exp2((ex - 1).to(D)), fr / 2)
        return torch.where(q > 7, -v, v) * torch.exp2(s.to(D) - 127).repeat_interleave(32, -1)

    def e4m3(q, s):
        q = q.to(torch.int32)
        ex, fr = q >> 3 & 15, (q & 7).to(D) / 8
        v = torch.where(ex > 0, (1 + fr) * torch.exp2((ex - 7).to(D)), fr * 2.0**-6)
        return torch.where(q > 127, -v, v) * torch.exp2(s.to(D) - 127).repeat_interleave(32, -1)

    def rms(v):
        return (v.square().mean(1, keepdim=True) + EPS) ** -0.5

    if op == "route":
        T, E, G, k = case["T"], case["E"], case["groups"], case["k"]
        lg = st["logits"].to(D).requires_grad_()
        if case["score"] == "sigmoid":
            s = 1 / (1 + torch.exp(-lg))
        else:
            s = torch.exp(lg - torch.logsumexp(lg, 1, keepdim=True))
        with torch.no_grad():
            by = s if st["bias"] is None else s + st["bias"].to(D)
            if G > 1:
                members = by.reshape(T, G, E // G).sort(dim=2).values.flip(2)[:, :, :case["top"]]
                value = members[:, :, 0]
                if members.shape[2] > 1:
                    value = value + torch.where(members[:, :, 1] > -math.inf, members[:, :, 1], 0.0)
                last = value.sort(dim=1).values[:, G - case["kept"]].unsqueeze(1)
                by = torch.where((value >= last).repeat_interleave(E // G, 1), by, -math.inf)
            idx = by.topk(k, dim=1).indices
            live = (by.gather(1, idx) > -math.inf).to(D)
        p = s.gather(1, idx) * live
        w = case["scale"] * (p / p.sum(1, keepdim=True) if case["renorm"] else p)
        out = {"idx": None, "w": w.detach(), "counts": None, "offsets": None, "row_of": None, "src_of": None}
        if case["bwd"]:
            (out["dlogits"],) = torch.autograd.grad((w * st["ds"].to(D)).sum(), lg)
        return out
    if op == "quant":
        v = st["v"].to(D)
        if case["col"]:
            v = v.mT.contiguous()
        b = v.unflatten(-1, (-1, 32))
        scale = torch.exp2(torch.ceil(torch.log2(b.abs().amax(-1, keepdim=True).clamp(min=2.0**-124) / 6)))
        t = b / scale
        step = torch.exp2(torch.floor(torch.log2(t.abs().clamp(min=1.0))) - 1)
        return {"v": (torch.round(t / step) * step * scale).flatten(-2), "s": None}
    if op == "experts":
        K, N, act = case["K"], case["N"], case["act"]
        x = st["x"].to(D) if case["x"] == "bf16" else e4m3(st["x"], st["x_s"]) if case["x"] == "mxfp8" else e2m1(st["x"], st["x_s"])
        y = torch.zeros(len(st["src_of"]), N // 2 if act in GATED else N, dtype=D, device="cuda")
        of_token = st["src_of"].long() // case["k"]
        i = torch.arange(N, device="cuda")
        for e in range(case["E"]):
            a, n = st["plan"][e]
            if n == 0:
                continue
            part = x[of_token[a:a + n]] if case["gather"] else x[a:a + n]
            z = part @ e2m1(st["w_q"][e], st["w_s"][e]).t()
            if act in GATED:
                h, u = z[:, i // 32 % 2 == 0], z[:, i // 32 % 2 == 1]
                z = (h / (1 + torch.exp(-h)) if act == "swiglu" else h * torch.special.ndtr(h)) * u
            y[a:a + n] = z
        return {"y": y}
    if op == "norm":
        x, w = st["x"].to(D), st["w"].to(D).requires_grad_()
        out = {}
        if case["res"]:
            out["total"] = x + st["res"].to(D)
            x = out["total"].to(torch.bfloat16).to(D)
        x.requires_grad_()
        r = rms(x)
        y = x * r * w
        out["y"], out["rstd"] = y.detach(), r.detach().squeeze(1)
        if case["bwd"]:
            dx, out["dw"] = torch.autograd.grad(y, (x, w), st["dy"].to(D))
            out["dx"] = dx + st["dres"].to(D)
        return {key: out[key] for key in ("total", "y", "rstd", "dx", "dw") if key in out}
    out, k = {}, case["k"]
    y, w = st["y"].to(D), st["w"].to(D).requires_grad_()
    if k:
        total = torch.zeros(case["T"], case["d"], dtype=D, device="cuda")
        for j in range(k):
            total += y[st["row_of"].long()[j::k]] * st["topk_w"][:, j:j + 1].to(D)
        out["total"] = total
        y = total.to(torch.bfloat16).to(D)
    gate = None if st["gate"] is None else st["gate"].to(D).requires_grad_()

    def block(v):
        branch = v * rms(v) * w
        if gate is not None:
            branch = branch * (1 / (1 + torch.exp(-gate)) if case["sigmoid"] else gate)
        return st["x"].to(D) + case["scale"] * branch

    out["out"], out["rstd"] = block(y).detach(), rms(y).squeeze(1)
    if case["bwd"]:
        y = st["saved"].to(D).requires_grad_()
        o = block(y)
        leaves = [y, w] + ([] if gate is None else [gate])
        grads = torch.autograd.grad(o, leaves, st["dout"].to(D))
        if gate is not None:
            out["dgate"] = grads[2]
        out["dy"], out["dw"] = grads[:2]
    return out
