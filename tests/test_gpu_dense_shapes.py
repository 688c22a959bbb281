"""The dense operators over seeded random shapes, with guard values around every output (GPU).

The reference is the same computation in 64 bits on the same bf16 inputs; bounds as in
test_gpu_dense: a sum of K products is off by at most K 2^-24 of the sum of magnitudes,
rounding to bf16 adds 2^-8, and the tests here take identity or squared ReLU, whose values
and slopes are exact to 2^-23.
"""
import random

import pytest
import torch

pytestmark = pytest.mark.gpu
U, H = 2.0**-24, 2.0**-8
BF, GUARD = torch.bfloat16, 4096


@pytest.fixture(scope="module")
def M():
    from ragged_grouped_gemm_device_amd import moe
    moe.load()
    return moe


class Guarded:
    """A tensor between two runs of guard values."""

    def __init__(self, shape, dtype):
        n = 1
        for s in shape:
            n *= s
        self.all = torch.full((n + 2 * GUARD,), 77, dtype=dtype, device="cuda")
        self.t = self.all[GUARD:GUARD + n].view(shape)

    def whole(self):
        return bool((self.all[:GUARD] == 77).all()) and bool((self.all[-GUARD:] == 77).all())


def _close(got, ref, bound, what):
    bad = ~((got.double() - ref).abs() <= bound + 2.0**-120)
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:3].tolist())


# shapes for which each tile form (and its split) is chosen for one of the three products
CHOSEN = [(5000, 3000, 1000), (600, 4096, 8192), (136, 3000, 4160), (3001, 4160, 136), (1030, 1544, 2880),
          (2048, 2048, 2048), (4096, 2048, 4096), (1020, 2880, 5760), (2300, 4096, 2304), (1100, 2056, 1152),
          (1500, 1032, 2112), (4100, 136, 1088), (20, 4168, 4104), (300, 4096, 64), (600, 8192, 8192),
          (6000, 4200, 4104), (4200, 4200, 6000), (4300, 4104, 4168), (4996, 4000, 4160)]


def _shape(rng, i):
    if i >= 48:
        return CHOSEN[i - 48]
    log = lambda lo, hi, step: max(step, int(lo * (hi / lo) ** rng.random()) // step * step)  # noqa: E731
    if i % 4 == 0:
        return log(1, 80, 1), log(8, 6000, 8), log(8, 6000, 8)       # few rows
    if i % 4 == 1:
        return log(2000, 20000, 1), log(8, 300, 8), log(8, 300, 8)   # many rows, narrow
    return log(8, 3000, 1), log(8, 3000, 8), log(8, 3000, 8)


@pytest.mark.parametrize("i", range(48 + len(CHOSEN)))
def test_random_shapes(M, i):
    rng = random.Random(i)
    T, K, N = _shape(rng, i)
    rng.random()
    act, srelu = ("srelu", True) if rng.random() < 0.5 else ("none", False)
    print(f"shape {i}: T={T} K={K} N={N} act={act}", flush=True)
    g = torch.Generator("cuda").manual_seed(i)
    new = lambda *s, std=1.0: (torch.randn(*s, device="cuda", generator=g) * std).to(BF)  # noqa: E731
    x, w, b, r, dy = new(T, K), new(K, N, std=K**-0.5), new(N), new(T, N), new(T, N)
    xd, wd, bd, rd, dyd = (t.double() for t in (x, w, b, r, dy))
    ws = Guarded((max(16, M.moe_linear_workspace_bytes(T, K, N)),), torch.uint8)
    outs = [ws]

    def out(shape, dtype):
        outs.append(Guarded(shape, dtype))
        return outs[-1].t

    code = M.MOE_ACT_SRELU if srelu else M.MOE_ACT_NONE
    y, y32 = out((T, N), BF), out((T, N), torch.float32)
    z = out((T, N), BF) if srelu else None
    mx = srelu and N % 32 == 0
    zq = out((T, N), torch.uint8) if mx else None
    zs = out((T, N // 32), torch.uint8) if mx else None
    M.moe_linear_fwd(x, w, y, code, b, r, z=z, z_q=zq, z_s=zs, workspace=ws.t)
    M.moe_linear_fwd(x, w, y32, code, b, workspace=ws.t)
    z0 = xd @ wd + bd
    zb = (K + 2) * U * (xd.abs() @ wd.abs() + bd.abs())
    f0 = z0.clamp(min=0).square() if srelu else z0
    fb = (2 * z0.abs() + zb) * zb + 4 * U * f0.abs() if srelu else zb
    _close(y32, f0, fb + U * f0.abs(), "y fp32")
    yb = fb + U * (f0.abs() + rd.abs())
    _close(y, f0 + rd, yb + H * ((f0 + rd).abs() + yb), "y")
    if srelu:
        _close(z, z0, zb + H * (z0.abs() + zb), "z")
        zq2, zs2 = out((T, N), torch.uint8) if mx else None, out((T, N // 32), torch.uint8) if mx else None
        if mx:
            M.moe_quant_mxfp8(z, M.MOE_QUANT_ROWWISE, zq2, zs2)
            assert torch.equal(zq, zq2) and torch.equal(zs, zs2)

    dz, db = out((T, N), BF), out((N,), torch.float32)
    if srelu:
        zv = z.double()
        if mx:
            back = out((T, N), BF)
            M.moe_dequant_mxfp8(zq, zs, back)
            zv = back.double()
        M.moe_act_bwd(dy, dz, code, z=None if mx else z, z_q=zq, z_s=zs, dbias=db, workspace=ws.t)
        ref = dyd * 2 * zv.clamp(min=0)
    else:
        M.moe_act_bwd(dy, dz, code, dbias=db, workspace=ws.t)
        ref = dyd
    _close(dz, ref, H * ref.abs() * (1 + 4 * U) + 4 * U * ref.abs(), "dz")
    _close(db, ref.sum(0), (T + 4) * U * ref.abs().sum(0), "dbias")

    dzd = dz.double()
    dx, dw, dwb = out((T, K), BF), out((K, N), torch.float32), out((K, N), BF)
    M.moe_linear_dgrad(dz, w, dx, residual=x, workspace=ws.t)
    ref = dzd @ wd.t() + xd
    bound = (N + 2) * U * (dzd.abs() @ wd.abs().t()) + 2 * U * xd.abs()
    _close(dx, ref, bound + H * (ref.abs() + bound), "dx")
    M.moe_linear_wgrad(x, dz, dw, workspace=ws.t)
    M.moe_linear_wgrad(x, dz, dwb, workspace=ws.t)
    ref, bound = xd.t() @ dzd, (T + 2) * U * (xd.abs().t() @ dzd.abs())
    _close(dw, ref, bound, "dw")
    _close(dwb, ref, bound + H * (ref.abs() + bound), "dw bf16")
    if K % 32 == 0:
        xq, xs, xb = out((T, K), torch.uint8), out((T, K // 32), torch.uint8), out((T, K), BF)
        M.moe_quant_mxfp8(x, M.MOE_QUANT_ROWWISE, xq, xs)
        M.moe_dequant_mxfp8(xq, xs, xb)
        M.moe_linear_wgrad(None, dz, dw, x_q=xq, x_s=xs, workspace=ws.t)
        x8 = xb.double()
        _close(dw, x8.t() @ dzd, (T + 2) * U * (x8.abs().t() @ dzd.abs()), "dw from the checkpoint")
    torch.cuda.synchronize()
    for o in outs:
        assert o.whole(), tuple(o.t.shape)


@pytest.mark.parametrize("i", range(16))
def test_random_losses_keep_to_their_buffers(M, i):
    rng = random.Random(100 + i)
    E = rng.choice([rng.randint(1, 1024), 1 << rng.randint(0, 10)])
    T = int(3000 ** rng.random()) + rng.randint(0, 3)
    k, S = rng.randint(1, min(E, 8)), rng.randint(1, max(1, min(T, 40)))
    T = max(T, S)
    print(f"losses {i}: T={T} E={E} k={k} S={S}", flush=True)
    g = torch.Generator("cuda").manual_seed(i)
    lg = torch.randn(T, E, device="cuda", generator=g)
    idx = lg.topk(k, 1).indices.to(torch.int32)
    seq = torch.randint(0, T + 1, (S + 1,), device="cuda", generator=g).sort().values.to(torch.int32)
    outs = {n: Guarded(s, d) for n, s, d in (
        ("loss", (3,), torch.float32), ("counts", (S, E), torch.int32), ("prob", (S, E), torch.float32),
        ("tokens", (S + 2,), torch.int32), ("d", (T, E), torch.float32), ("d16", (T, E), BF),
        ("ws", (M.moe_balance_workspace_bytes(T, E, S),), torch.uint8))}
    o = {n: v.t for n, v in outs.items()}
    M.moe_balance_loss(lg, idx, o["loss"], o["counts"], o["prob"], o["tokens"], o["ws"], 1.0, 0.5, seq_offsets=seq)
    M.moe_balance_loss_bwd(lg, o["counts"], o["tokens"], o["d"], k, 1.0, 0.5, seq_offsets=seq, dlogits_bf16=o["d16"])
    torch.cuda.synchronize()
    for n, v in outs.items():
        assert v.whole(), n
    lo, hi = int(seq[0]), int(seq[-1])
    assert int(o["tokens"][S + 1]) == hi - lo
    assert int(o["counts"].sum()) == (hi - lo) * k
    assert not o["d"][:lo].any() and not o["d"][hi:].any()
    assert torch.equal(o["d16"], o["d"].to(BF))
    # the gradient of a token sums to that of its z term: sum_e p_e (f_e - sum f p) = 0
    lse = torch.logsumexp(lg[lo:hi].double(), 1)
    want = 0.5 * 2 * lse / max(hi - lo, 1)
    got = o["d"][lo:hi].double().sum(1)
    scale = o["d"][lo:hi].double().abs().sum(1)
    assert ((got - want).abs() <= 2.0**-16 * (scale + want.abs()) + 1e-30).all()


@pytest.mark.parametrize("T, K, N", CHOSEN)
def test_gated_epilogue_of_every_tile_form(M, T, K, N):
    """SwiGLU with bias, residual and 8-bit checkpoint where each tile form runs: z against 64 bits,
    y against f of the fp32 sums (f and its slope in g are bounded by |g| and 1.1; the exponential is
    off by (2 |g| + 2) 2^-23), codes against the quantizer."""
    N = N // 64 * 64
    g = torch.Generator("cuda").manual_seed(T)
    new = lambda *s, std=1.0: (torch.randn(*s, device="cuda", generator=g) * std).to(BF)  # noqa: E731
    x, w, b, r = new(T, K), new(K, N, std=K**-0.5), new(N), new(T, N // 2)
    y, z = Guarded((T, N // 2), BF), Guarded((T, N), BF)
    zq, zs = Guarded((T, N), torch.uint8), Guarded((T, N // 32), torch.uint8)
    ws = Guarded((max(16, M.moe_linear_workspace_bytes(T, K, N)),), torch.uint8)
    M.moe_linear_fwd(x, w, y.t, M.MOE_ACT_SWIGLU, b, r, z=z.t, z_q=zq.t, z_s=zs.t, workspace=ws.t)
    q, s = torch.empty_like(zq.t), torch.empty_like(zs.t)
    M.moe_quant_mxfp8(z.t, M.MOE_QUANT_ROWWISE, q, s)
    torch.cuda.synchronize()
    assert all(o.whole() for o in (y, z, zq, zs, ws))
    assert torch.equal(q, zq.t) and torch.equal(s, zs.t)
    z0 = x.double() @ w.double() + b.double()
    zb = (K + 2) * U * (x.double().abs() @ w.double().abs() + b.double().abs())
    _close(z.t, z0, zb + H * (z0.abs() + zb), "z")
    halves = lambda v: [v.reshape(T, -1, 2, 32)[:, :, j].reshape(T, -1) for j in (0, 1)]  # noqa: E731
    (gt, up), (gb, ub) = halves(z0), halves(zb)
    f = gt * torch.sigmoid(gt)
    fb = 1.2 * gb + (2 * gt.abs() + 8) * 2 * U * gt.abs()
    ref = f * up + r.double()
    bound = fb * (up.abs() + ub) + f.abs() * ub + 4 * U * (f * up).abs() + 2 * U * r.double().abs()
    _close(y.t, ref, bound + H * (ref.abs() + bound), "y")
