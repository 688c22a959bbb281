"""Cases of the dense half of a mixture-of-experts layer: the linear layer of a
shared expert or a router projection (bias, activation and residual in the
product's epilogue, its pre-activation kept as an 8-bit checkpoint), its
backward pass from 8-bit checkpoints, the router's balance and z losses with
their gradient, and the restoring of an 8-bit checkpoint.

Weights are [in, out] row-major; a gated layer's columns hold 32 gate columns
and 32 up columns in turn. An 8-bit checkpoint holds E4M3 codes and one E8M0
scale for 32 neighbouring columns of a row: the smallest power of two that
keeps the block's largest bf16 magnitude within 448.
"""
import math

import torch

own = False

GATED = ("swiglu", "geglu")


def listed():
    return [
        # one token through a shared expert's gate/up projection: latency
        {"name": "linear-one-token", "op": "linear", "T": 1, "K": 8192, "N": 4096, "act": "swiglu", "bias": False, "res": False, "save": "", "f32": False},
        # a decode batch through its down projection, added to the routed experts' output
        {"name": "linear-decode-down", "op": "linear", "T": 24, "K": 2048, "N": 7168, "act": "none", "bias": False, "res": True, "save": "", "f32": False},
        # router logits of a prompt: a narrow product with a float32 result
        {"name": "linear-router-logits", "op": "linear", "T": 4096, "K": 7168, "N": 32, "act": "none", "bias": False, "res": False, "save": "", "f32": True},
        # a ragged micro-batch of a 2880-wide model, biased GeGLU, 8-bit checkpoint
        {"name": "linear-odd-rows", "op": "linear", "T": 1000, "K": 2880, "N": 5760, "act": "geglu", "bias": True, "res": False, "save": "mx", "f32": False},
        # a training step's tokens through a shared expert's gate/up projection, 8-bit checkpoint
        {"name": "linear-train", "op": "linear", "T": 32768, "K": 8192, "N": 4096, "act": "swiglu", "bias": False, "res": False, "save": "mx", "f32": False},
        # backward of the ragged micro-batch: input and pre-activation from 8-bit checkpoints
        {"name": "backward-odd-rows", "op": "backward", "T": 1000, "K": 2880, "N": 5760, "act": "geglu", "bias": True, "x8": True, "z8": True, "f32": False},
        # backward of a down projection (no activation), float32 weight gradient
        {"name": "backward-down", "op": "backward", "T": 4096, "K": 2048, "N": 7168, "act": "none", "bias": False, "x8": False, "z8": False, "f32": True},
        # backward of a training step's gate/up projection from 8-bit checkpoints
        {"name": "backward-train", "op": "backward", "T": 16384, "K": 7168, "N": 4096, "act": "swiglu", "bias": False, "x8": True, "z8": True, "f32": False},
        # router losses of a small batch: launches count
        {"name": "balance-small", "op": "balance", "T": 256, "E": 8, "k": 2, "S": 1, "mask": False},
        # router losses per sequence over a packed batch with padding tokens
        {"name": "balance-sequences", "op": "balance", "T": 131072, "E": 256, "k": 8, "S": 64, "mask": True},
        # one expert's rows of a checkpoint restored for the backward pass
        {"name": "restore-small", "op": "restore", "R": 1021, "C": 2880},
        # a training step's checkpointed expert pre-activations restored
        {"name": "restore-train", "op": "restore", "R": 32768, "C": 4096},
    ]


def _log(rng, lo, hi, step=1):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(lo, min(hi, v // step * step))


def draw(rng):
    op = rng.choice(["linear", "linear", "backward", "backward", "balance", "restore"])
    if op == "restore":
        return {"op": op, "R": _log(rng, 1, 32768), "C": _log(rng, 32, 4096, 32)}
    if op == "balance":
        E = rng.choice([_log(rng, 2, 256), 1 << rng.randint(3, 8)])
        T = _log(rng, 1, 131072)
        return {"op": op, "T": T, "E": E, "k": rng.randint(1, min(8, E)), "S": min(T, _log(rng, 1, 64)),
                "mask": rng.random() < 0.5}
    act = rng.choice(["swiglu", "geglu", "none", "silu", "gelu", "srelu"])
    step = 64 if act in GATED else rng.choice([8, 32])
    T, K, N = _log(rng, 1, 32768), _log(rng, 64, 8192, 8), _log(rng, 64, 8192, step)
    most = 32768 * 8192 * 4096 if op == "linear" else 16384 * 7168 * 4096
    if T * K * N > most:
        T = most // (K * N)
    if op == "linear":
        f32 = act == "none" and rng.random() < 0.3
        save = rng.choice(["", "mx" if N % 32 == 0 else "", "bf16"]) if act != "none" else ""
        return {"op": op, "T": T, "K": K, "N": N, "act": act, "bias": rng.random() < 0.5, "res": rng.random() < 0.4,
                "save": save, "f32": f32}
    return {"op": op, "T": T, "K": K, "N": N, "act": act, "bias": rng.random() < 0.5, "x8": K % 32 == 0 and rng.random() < 0.6,
            "z8": act != "none" and N % 32 == 0 and rng.random() < 0.7, "f32": act == "none"}


# ---------------------------------------------------------------- 8-bit blocks
def _to_mx(v):
    """Codes and scales of a float32 or float64 matrix, of its bf16 values."""
    b = v.to(torch.bfloat16).float().reshape(v.shape[0], -1, 32)
    m, x = torch.frexp(b.abs().amax(2))  # amax = m 2^x, m in [0.5, 1)
    e = torch.where(m > 0.875, x - 8, x - 9).clamp(-127, 127)  # 448 = 0.875 * 2^9
    e = torch.where(m == 0, torch.full_like(e, -127), e)
    q = torch.ldexp(b, -e.unsqueeze(2)).to(torch.float8_e4m3fn).view(torch.uint8)
    return q.reshape(v.shape), (e + 127).to(torch.uint8)


def _from_mx(q, s, dtype=torch.float32):
    v = q.view(torch.float8_e4m3fn).to(dtype).reshape(q.shape[0], -1, 32)
    return torch.ldexp(v, s.to(torch.int32).unsqueeze(2) - 127).reshape(q.shape)


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, device="cuda", generator=g) * std).to(torch.bfloat16)

    st = {"case": case}
    if case["op"] == "linear":
        T, K, N = case["T"], case["K"], case["N"]
        out = N // 2 if case["act"] in GATED else N
        st["x"], st["w"] = normal(T, K), normal(K, N, std=0.02)
        st["bias"] = normal(N, std=0.5) if case["bias"] else None
        st["res"] = normal(T, out) if case["res"] else None
    elif case["op"] == "backward":
        T, K, N = case["T"], case["K"], case["N"]
        out = N // 2 if case["act"] in GATED else N
        st["w"], st["dy"] = normal(K, N, std=0.02), normal(T, out)
        x = normal(T, K)
        st["x"], st["x8"] = (None, _to_mx(x.float())) if case["x8"] else (x, None)
        st["z"] = st["z8"] = None
        if case["act"] != "none":
            z = normal(T, N, std=0.02 * math.sqrt(K))
            st["z"], st["z8"] = (None, _to_mx(z.float())) if case["z8"] else (z, None)
    elif case["op"] == "balance":
        T, E, k, S = case["T"], case["E"], case["k"], case["S"]
        popular = torch.randperm(E, device="cuda", generator=g) + 1  # a few experts are asked for more
        st["logits"] = torch.randn(T, E, device="cuda", generator=g) - 0.5 * popular.log()
        st["idx"] = st["logits"].topk(k, dim=1).indices.to(torch.int32)
        cuts = torch.randint(0, T + 1, (S - 1,), device="cuda", generator=g).sort().values
        ends = [torch.zeros(1, device="cuda", dtype=torch.int64), cuts, torch.full((1,), T, device="cuda")]
        st["seq"] = torch.cat(ends).to(torch.int32) if S > 1 else None
        st["valid"] = (torch.rand(T, device="cuda", generator=g) < 0.9).to(torch.uint8) if case["mask"] else None
    else:
        R, C = case["R"], case["C"]
        mag = torch.randint(0, 127, (R, C), device="cuda", generator=g, dtype=torch.int32)  # 127 is NaN
        sign = torch.randint(0, 2, (R, C), device="cuda", generator=g, dtype=torch.int32) * 128
        st["q"] = (mag + sign).to(torch.uint8)
        st["s"] = torch.randint(110, 131, (R, C // 32), device="cuda", generator=g, dtype=torch.int32).to(torch.uint8)
    return st


BALANCE_COEF, Z_COEF = 1e-2, 1e-3  # usual weights of the two router losses


# ---------------------------------------------------------------- plain forms
def _phi(g):
    return 0.5 * (1 + torch.erf(g * math.sqrt(0.5)))


def _act(z, act):
    if act == "none":
        return z
    if act == "srelu":
        return z.clamp(min=0).square()
    if act in GATED:
        h = z.reshape(z.shape[0], -1, 2, 32)
        return (_act(h[:, :, 0], "silu" if act == "swiglu" else "gelu") * h[:, :, 1]).reshape(z.shape[0], -1)
    return z * torch.sigmoid(z) if act == "silu" else z * _phi(z)


def _act_slope(z, act):
    if act == "srelu":
        return 2 * z.clamp(min=0)
    if act == "silu":
        s = torch.sigmoid(z)
        return s * (1 + z * (1 - s))
    return _phi(z) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)


def _dz(dy, z, act):
    if act == "none":
        return dy
    if act in GATED:
        inner = "silu" if act == "swiglu" else "gelu"
        h, d = z.reshape(z.shape[0], -1, 2, 32), dy.reshape(z.shape[0], -1, 32)
        gate = d * h[:, :, 1] * _act_slope(h[:, :, 0], inner)
        return torch.stack((gate, d * _act(h[:, :, 0], inner)), 2).reshape(z.shape)
    return dy * _act_slope(z, act)


def _plain(st):
    c = st["case"]
    if c["op"] == "linear":
        z = st["x"].float() @ st["w"].float()
        if st["bias"] is not None:
            z = z + st["bias"].float()
        y = _act(z, c["act"])
        if st["res"] is not None:
            y = y + st["res"].float()
        out = {"y": y if c["f32"] else y.to(torch.bfloat16)}
        if c["save"]:
            out["z"] = (_from_mx(*_to_mx(z)) if c["save"] == "mx" else z).to(torch.bfloat16)
        return out
    if c["op"] == "backward":
        z = _from_mx(*st["z8"]) if st["z8"] is not None else st["z"].float() if st["z"] is not None else None
        x = _from_mx(*st["x8"]) if st["x8"] is not None else st["x"].float()
        dz = _dz(st["dy"].float(), z, c["act"])
        out = {"dx": (dz @ st["w"].float().t()).to(torch.bfloat16)}
        dw = x.t() @ dz
        out["dw"] = dw if c["f32"] else dw.to(torch.bfloat16)
        if c["bias"]:
            out["dbias"] = dz.sum(0)
        return out
    if c["op"] == "balance":
        return _balance_plain(st)
    return {"v": _from_mx(st["q"], st["s"]).to(torch.bfloat16)}


def _balance_plain(st):
    lg, idx, c = st["logits"], st["idx"], st["case"]
    T, E, k, S = c["T"], c["E"], c["k"], c["S"]
    valid = torch.ones(T, device=lg.device) if st["valid"] is None else (st["valid"] != 0).float()
    if st["seq"] is None:
        seq = torch.zeros(T, dtype=torch.int64, device=lg.device)
    else:
        seq = torch.searchsorted(st["seq"][1:], torch.arange(T, device=lg.device, dtype=torch.int32), right=True)
    top = lg.amax(1, keepdim=True)
    ex = torch.exp(lg - top)
    total = ex.sum(1, keepdim=True)
    p, lse = ex / total, (torch.log(total) + top).squeeze(1)
    member = (seq == torch.arange(S, device=lg.device).unsqueeze(1)) * valid  # [S, T]: sequence s owns a live token t
    n = member.sum(1)
    live = (n > 0).float().sum().clamp(min=1)
    count = member @ torch.zeros(T, E, device=lg.device).scatter_add_(1, idx.long(), torch.ones_like(idx, dtype=torch.float32))
    mean = member.double() @ p.double()
    per = n.clamp(min=1).unsqueeze(1)
    mean, f = (mean / per).float(), count * E / (k * per)
    balance = (f * mean).double().sum().float() / live
    many = valid.sum().clamp(min=1)
    z = (valid * lse.square()).double().sum().float() / many
    loss = torch.stack((BALANCE_COEF * balance + Z_COEF * z, balance, z))
    # f less its value at the largest logit: no cancellation where one expert has all the probability
    fs = f[seq] - f[seq, lg.argmax(1)].unsqueeze(1)
    db = p * (fs - (p * fs).sum(1, keepdim=True)) * (BALANCE_COEF / live / per[seq])
    dl = (db + p * (2 * Z_COEF * lse / many).unsqueeze(1)) * valid.unsqueeze(1)
    return {"loss": loss, "counts": count.to(torch.int32), "prob": mean, "dlogits": dl}


# ---------------------------------------------------------------- the framework's operators
def _own(st):
    from ragged_grouped_gemm_device_amd import moe as M

    c = st["case"]
    acts = {"swiglu": M.MOE_ACT_SWIGLU, "geglu": M.MOE_ACT_GEGLU, "srelu": M.MOE_ACT_SRELU,
            "none": M.MOE_ACT_NONE, "silu": M.MOE_ACT_SILU, "gelu": M.MOE_ACT_GELU}
    bf, f32, i32, u8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
    if "buf" not in st:  # outputs and workspace, allocated once and kept as a training or serving loop keeps them
        st["buf"] = b = {}

        def new(name, dtype, *shape):
            b[name] = torch.empty(*shape, dtype=dtype, device="cuda")

        if c["op"] == "linear":
            T, K, N = c["T"], c["K"], c["N"]
            new("y", f32 if c["f32"] else bf, T, N // 2 if c["act"] in GATED else N)
            if c["save"]:
                new("z", bf, T, N)
            if c["save"] == "mx":
                new("z_q", u8, T, N)
                new("z_s", u8, T, N // 32)
            new("ws", u8, max(16, M.moe_linear_workspace_bytes(T, K, N, M.MOE_LINEAR_FWD)))
        elif c["op"] == "backward":
            T, K, N = c["T"], c["K"], c["N"]
            if c["act"] != "none":
                new("dz", bf, T, N)
            new("dx", bf, T, K)
            new("dw", f32 if c["f32"] else bf, K, N)
            if c["bias"]:
                new("dbias", f32, N)
            new("ws", u8, max(16, M.moe_linear_workspace_bytes(T, K, N, M.MOE_LINEAR_BWD)))
        elif c["op"] == "balance":
            T, E, S = c["T"], c["E"], c["S"]
            new("loss", f32, 3)
            new("counts", i32, S, E)
            new("prob", f32, S, E)
            new("tokens", i32, S + 2)
            new("dlogits", f32, T, E)
            new("ws", u8, max(16, M.moe_balance_workspace_bytes(T, E, S)))
        else:
            new("v", bf, c["R"], c["C"])
    b = st["buf"]
    if c["op"] == "linear":
        mx = c["save"] == "mx"
        M.moe_linear_fwd(st["x"], st["w"], b["y"], act=acts[c["act"]], bias=st["bias"], residual=st["res"],
                         z=None if mx else b.get("z"), z_q=b.get("z_q"), z_s=b.get("z_s"), workspace=b["ws"])
        if not c["save"]:
            return {"y": b["y"]}
        if mx:
            M.moe_dequant_mxfp8(b["z_q"], b["z_s"], b["z"])
        return {"y": b["y"], "z": b["z"]}
    if c["op"] == "backward":
        zq, zs = st["z8"] or (None, None)
        xq, xs = st["x8"] or (None, None)
        dz = st["dy"] if c["act"] == "none" else b["dz"]
        if c["act"] != "none" or c["bias"]:
            M.moe_act_bwd(st["dy"], b.get("dz"), act=acts[c["act"]], z=st["z"], z_q=zq, z_s=zs,
                          dbias=b.get("dbias"), workspace=b["ws"])
        M.moe_linear_dgrad(dz, st["w"], b["dx"], workspace=b["ws"])
        M.moe_linear_wgrad(st["x"], dz, b["dw"], x_q=xq, x_s=xs, workspace=b["ws"])
        return {key: b[key] for key in ("dx", "dw", "dbias") if key in b}
    if c["op"] == "balance":
        M.moe_balance_loss(st["logits"], st["idx"], b["loss"], b["counts"], b["prob"], b["tokens"], b["ws"],
                           BALANCE_COEF, Z_COEF, valid=st["valid"], seq_offsets=st["seq"])
        M.moe_balance_loss_bwd(st["logits"], b["counts"], b["tokens"], b["dlogits"], c["k"],
                               BALANCE_COEF, Z_COEF, valid=st["valid"], seq_offsets=st["seq"])
        return {key: b[key] for key in ("loss", "counts", "prob", "dlogits")}
    M.moe_dequant_mxfp8(st["q"], st["s"], b["v"])
    return {"v": b["v"]}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- least work
def work(case):
    if case["op"] == "linear":
        T, K, N = case["T"], case["K"], case["N"]
        out = N // 2 if case["act"] in GATED else N
        nbytes = 2 * (T * K + K * N + (N if case["bias"] else 0) + (T * out if case["res"] else 0)) + T * out * (4 if case["f32"] else 2)
        nbytes += {"": 0, "bf16": 2 * T * N, "mx": T * N + T * N // 32}[case["save"]]
        return {"bytes": nbytes, "flops": 2 * T * K * N}
    if case["op"] == "backward":
        T, K, N = case["T"], case["K"], case["N"]
        out = N // 2 if case["act"] in GATED else N
        x = T * K + T * K // 32 if case["x8"] else 2 * T * K
        z = 0 if case["act"] == "none" else T * N + T * N // 32 if case["z8"] else 2 * T * N
        return {"bytes": x + z + 2 * T * out + 2 * K * N + 2 * T * K + K * N * (4 if case["f32"] else 2) + (4 * N if case["bias"] else 0),
                "flops": 4 * T * K * N}
    if case["op"] == "balance":
        T, E, k, S = case["T"], case["E"], case["k"], case["S"]
        return {"bytes": 8 * T * E + 4 * T * k + (T if case["mask"] else 0) + 8 * S * E, "flops": 12 * T * E}
    return {"bytes": case["R"] * case["C"] * 3 + case["R"] * case["C"] // 32, "flops": 0}


# ---------------------------------------------------------------- 64-bit values
def exact(case, seed):
    st = prepare(case, seed)
    D = torch.float64

    def gate(v, act):
        return v / (1 + torch.exp(-v)) if act in ("silu", "swiglu") else v * torch.special.ndtr(v)

    def slope(v, act):
        if act in ("silu", "swiglu"):
            e = torch.exp(-v.abs())
            return (torch.where(v >= 0, 1.0, e) + v * e / (1 + e)) / (1 + e)
        return torch.special.ndtr(v) + v * torch.exp(-v * v / 2) / (2 * math.pi) ** 0.5

    def halves(v):  # gate and up columns of an interleaved matrix
        i = torch.arange(v.shape[1], device=v.device)
        return v[:, i // 32 % 2 == 0], v[:, i // 32 % 2 == 1]

    act = case.get("act")
    if case["op"] == "linear":
        z = st["x"].to(D) @ st["w"].to(D)
        if st["bias"] is not None:
            z += st["bias"].to(D)
        if act in GATED:
            a, u = halves(z)
            y = gate(a, act) * u
        elif act == "srelu":
            y = torch.where(z > 0, z * z, 0.0)
        else:
            y = z if act == "none" else gate(z, act)
        if st["res"] is not None:
            y = y + st["res"].to(D)
        if not case["save"]:
            return {"y": y}
        if case["save"] == "bf16":
            return {"y": y, "z": z}
        b = z.to(torch.bfloat16).to(D)
        most = b.abs().unflatten(1, (-1, 32)).amax(2).clamp(min=2.0**-118)
        scale = torch.exp2(torch.ceil(torch.log2(most / 448))).repeat_interleave(32, 1)
        t = b / scale
        step = torch.exp2(torch.floor(torch.log2(t.abs().clamp(min=2.0**-6))) - 3)
        return {"y": y, "z": torch.round(t / step) * step * scale}
    if case["op"] == "backward":
        def value(q, s):
            q = q.to(torch.int32)
            ex, fr = q >> 3 & 15, (q & 7).to(D) / 8
            v = torch.where(ex > 0, (1 + fr) * torch.exp2((ex - 7).to(D)), fr * 2.0**-6)
            return torch.where(q > 127, -v, v) * torch.exp2(s.to(D) - 127).repeat_interleave(32, 1)

        x = value(*st["x8"]) if case["x8"] else st["x"].to(D)
        dz = st["dy"].to(D)
        if act != "none":
            z = value(*st["z8"]) if case["z8"] else st["z"].to(D)
            if act in GATED:
                a, u = halves(z)
                i = torch.arange(z.shape[1], device=z.device)
                whole = torch.empty_like(z)
                whole[:, i // 32 % 2 == 0] = dz * u * slope(a, act)
                whole[:, i // 32 % 2 == 1] = dz * gate(a, act)
                dz = whole
            else:
                dz = dz * (torch.where(z > 0, 2 * z, 0.0) if act == "srelu" else slope(z, act))
        out = {"dx": dz @ st["w"].to(D).t(), "dw": x.t() @ dz}
        if case["bias"]:
            out["dbias"] = dz.sum(0)
        return out
    if case["op"] == "balance":
        E, k = case["E"], case["k"]
        lg = st["logits"].to(D).requires_grad_()
        live = torch.ones(case["T"], device="cuda", dtype=torch.bool) if st["valid"] is None else st["valid"] > 0
        ends = [0, case["T"]] if st["seq"] is None else st["seq"].tolist()
        p = torch.softmax(lg, 1)
        terms, means = [], []
        for a, b in zip(ends[:-1], ends[1:]):
            here = live[a:b]
            n = int(here.sum())
            if not n:
                means.append(torch.zeros(E, dtype=D, device="cuda"))
                continue
            asked = torch.bincount(st["idx"][a:b][here].reshape(-1).long(), minlength=E).to(D)
            means.append(p[a:b][here].mean(0))
            terms.append((asked * (E / (k * n)) * means[-1]).sum())
        zero = lg.sum() * 0
        balance = torch.stack(terms).mean() if terms else zero
        z = torch.logsumexp(lg[live], 1).square().mean() if terms else zero
        loss = BALANCE_COEF * balance + Z_COEF * z
        (d,) = torch.autograd.grad(loss, lg)
        return {"loss": torch.stack((loss, balance, z)).detach(), "counts": None, "prob": torch.stack(means).detach(), "dlogits": d}
    q, s = st["q"].to(torch.int32), st["s"].to(D)
    ex, fr = q >> 3 & 15, (q & 7).to(D) / 8
    v = torch.where(ex > 0, (1 + fr) * torch.exp2((ex - 7).to(D)), fr * 2.0**-6)
    return {"v": torch.where(q > 127, -v, v) * torch.exp2(s - 127).repeat_interleave(32, 1)}
