"""The norms around a block against the fp64 oracle (GPU).

Bounds: a bf16 result is off by half a step, 2^-8 of it at most (2^-9 and what follows for a rounding to
nearest), beside fp32 sums of n terms, n 2^-24 of the sum of their magnitudes; the row's statistics are
such sums of d terms, taken by threads of at most d / 64 each and joined in a tree: 64 2^-24 is ample."""
import numpy as np
import pytest
import torch

from oracle import block_oracle as B

from ._util import bf16_values

pytestmark = pytest.mark.gpu
EPS = 1e-5
HALF, SUM = 2.0**-8, 64 * 2.0**-24
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def M():
    from ragged_grouped_gemm_device_amd import moe
    moe.load()
    return moe


def rand(*shape, seed=0, std=1.0, mean=0.0):
    g = torch.Generator("cuda").manual_seed(seed + sum(shape))
    return (torch.randn(*shape, device="cuda", generator=g) * std + mean).to(BF)


def full(*shape, t=BF):
    return torch.full(shape, float("nan"), dtype=t, device="cuda")


def close(got, ref, slack, what):
    got = got.double().cpu().numpy().reshape(ref.shape)
    bad = np.abs(got - ref) > slack
    assert not bad.any(), (what, int(bad.sum()), float(np.abs(got - ref).max()))


SHAPES = [(1, 8), (3, 64), (5, 512), (6, 520), (1, 1024), (9, 1032), (130, 2048), (67, 2880), (1, 7168), (33, 8192), (5, 8200), (3, 16384),
          (1021, 64), (4500, 256)]


@pytest.mark.parametrize("T, d", SHAPES)
@pytest.mark.parametrize("res", [False, True])
def test_norm_and_its_gradient(M, T, d, res):
    x, w, dy = rand(T, d), rand(d, std=0.3, mean=1.0, seed=1), rand(T, d, seed=2)
    r, dres = (rand(T, d, seed=3), rand(T, d, seed=4)) if res else (None, None)
    total, y, rstd, dx, dw = full(T, d) if res else None, full(T, d), full(T, t=F32), full(T, d), full(d, t=F32)
    ws = torch.full((max(16, M.moe_norm_workspace_bytes(T, d)),), 255, dtype=torch.uint8, device="cuda")
    M.moe_norm_fwd(x, w, y, rstd, EPS, residual=r, total=total)
    s = x if not res else total
    if res:
        assert torch.equal(total, (x.float() + r.float()).to(BF))
    sv, wv, dv = bf16_values(s), bf16_values(w), bf16_values(dy)
    ref, rr = B.norm(sv, wv, EPS)
    close(rstd, rr, SUM * rr, "rstd")
    close(y, ref, (HALF + SUM) * np.abs(ref) + 1e-38, "y")
    M.moe_norm_bwd(dy, s, w, rstd, dx, dw, ws, dres=dres)
    rx, rw = B.norm_bwd(dv, sv, wv, EPS)
    terms = rr[:, None] * (np.abs(dv * wv) + np.abs(sv * rr[:, None]) * np.abs(dv * wv * sv * rr[:, None]).mean(1, keepdims=True))
    if res:
        rx = rx + bf16_values(dres)
        terms = terms + np.abs(bf16_values(dres))
    close(dx, rx, HALF * np.abs(rx) + 2 * SUM * terms, "dx")
    close(dw, rw, (T + 64) * 2.0**-24 * np.abs(dv * sv * rr[:, None]).sum(0) + 1e-30, "dw")
    alone = full(T, d)
    M.moe_norm_bwd(dy, s, w, rstd, alone, dres=dres)      # without dw: no workspace
    assert torch.equal(alone, dx)


@pytest.mark.parametrize("T, d, k", [(1, 64, 1), (7, 512, 4), (9, 1032, 2), (67, 2880, 8), (1, 7168, 8), (33, 8192, 3), (3, 16384, 2), (2000, 128, 2)])
@pytest.mark.parametrize("cols, sig", [(0, False), (1, True), (1, False), ("d", True), ("d", False)])
def test_post_norm_and_its_gradient(M, T, d, k, cols, sig):
    rows = T * k + 5
    cols = d if cols == "d" else cols
    Y, x, w, do = rand(rows, d), rand(T, d, seed=1), rand(d, std=0.3, mean=1.0, seed=2), rand(T, d, seed=3)
    row_of = torch.randperm(rows, device="cuda", generator=torch.Generator("cuda").manual_seed(T))[:T * k].to(torch.int32)
    tw = torch.rand(T, k, device="cuda", generator=torch.Generator("cuda").manual_seed(d))
    gate = rand(T, cols, seed=4, std=2.0) if cols else None
    act = M.MOE_GATE_SIGMOID if sig else M.MOE_GATE_LINEAR
    total, out, rstd = full(T, d), full(T, d), full(T, t=F32)
    M.moe_post_norm_fwd(Y, x, w, out, rstd, EPS, gate=gate, gate_act=act, scale=0.7, row_of=row_of, topk_w=tw, total=total)
    want = full(T, d)
    M.moe_combine(Y, row_of, tw, k, want)
    assert torch.equal(total, want)                      # bit for bit what the combination alone gives
    two, rstd2 = full(T, d), full(T, t=F32)
    M.moe_post_norm_fwd(total, x, w, two, rstd2, EPS, gate=gate, gate_act=act, scale=0.7)
    assert torch.equal(two, out) and torch.equal(rstd, rstd2)
    yv, xv, wv, dv = (bf16_values(t) for t in (total, x, w, do))
    gv = None if gate is None else bf16_values(gate)
    ref, rr = B.post_norm(yv, xv, wv, EPS, gv, sig, 0.7)
    branch = np.abs(ref - xv)
    close(rstd, rr, SUM * rr, "rstd")
    close(out, ref, HALF * np.abs(ref) + 2 * SUM * (branch + np.abs(xv)), "out")
    dy, dw = full(T, d), full(d, t=F32)
    dgate = None if gate is None else full(T, cols, t=F32 if cols == 1 else BF)
    ws = torch.full((max(16, M.moe_norm_workspace_bytes(T, d)),), 255, dtype=torch.uint8, device="cuda")
    M.moe_post_norm_bwd(do, total, w, rstd, dy, dw, ws, gate=gate, dgate=dgate, gate_act=act, scale=0.7)
    ry, rg, rw = B.post_norm_bwd(dv, yv, wv, EPS, gv, sig, 0.7)
    h = np.abs(yv * rr[:, None])
    f = np.ones((1, 1)) if gv is None else np.abs(1 / (1 + np.exp(-gv)) if sig else gv)
    g = 0.7 * np.abs(dv * wv) * f
    close(dy, ry, HALF * np.abs(ry) + 2 * SUM * rr[:, None] * (g + h * (g * h).mean(1, keepdims=True)), "dy")
    close(dw, rw, (T + 80) * 2.0**-24 * (0.7 * np.abs(dv) * f * h).sum(0) + 1e-30, "dw")
    if cols == 1:
        close(dgate, rg, 2 * SUM * (0.7 * np.abs(dv * wv) * h).sum(1, keepdims=True), "dgate")
    elif cols:
        close(dgate, rg, (HALF + SUM) * np.abs(rg) + 1e-38, "dgate")


def test_rows_keep_to_themselves(M):
    """A row of zeros, one with a NaN, one with an infinity: the others' results do not change."""
    T, d = 9, 2880
    x, w = rand(T, d), rand(d, seed=1)
    y, y2, rstd = full(T, d), full(T, d), full(T, t=F32)
    M.moe_norm_fwd(x, w, y, rstd, EPS)
    x2 = x.clone()
    x2[2], x2[4, 7], x2[6, 9] = 0, float("nan"), float("inf")
    M.moe_norm_fwd(x2, w, y2, rstd, EPS)
    keep = [0, 1, 3, 5, 7, 8]
    assert torch.equal(y[keep], y2[keep]) and (y2[2] == 0).all() and y2[4].isnan().all()
    assert abs(float(rstd[2]) - EPS**-0.5) <= SUM * EPS**-0.5


def test_outputs_that_are_inputs(M):
    """In place where the documentation allows it."""
    T, d = 37, 2880
    x, r, w, dy, dres = (rand(T, d, seed=i) if i != 2 else rand(d, seed=2) for i in range(5))
    t1, y1, rs = full(T, d), full(T, d), full(T, t=F32)
    M.moe_norm_fwd(x, w, y1, rs, EPS, residual=r, total=t1)
    for which in (0, 1):
        xi, ri, y2 = x.clone(), r.clone(), full(T, d)
        M.moe_norm_fwd(xi, w, y2, None, EPS, residual=ri, total=(xi, ri)[which])
        assert torch.equal((xi, ri)[which], t1) and torch.equal(y2, y1)
    y0, xi = full(T, d), x.clone()
    M.moe_norm_fwd(x, w, y0, None, EPS)
    M.moe_norm_fwd(xi, w, xi, None, EPS)
    assert torch.equal(xi, y0)
    dx = full(T, d)
    M.moe_norm_bwd(dy, t1, w, rs, dx, dres=dres)
    for which in (0, 1):
        a, b = dy.clone(), dres.clone()
        M.moe_norm_bwd(a, t1, w, rs, (a, b)[which], dres=b)
        assert torch.equal((a, b)[which], dx)
    out, xi, gate = full(T, d), x.clone(), rand(T, d, seed=9)
    M.moe_post_norm_fwd(r, x, w, out, None, EPS, gate=gate)
    M.moe_post_norm_fwd(r, xi, w, xi, None, EPS, gate=gate)
    assert torch.equal(xi, out)
    a, d1 = dy.clone(), full(T, d)
    M.moe_post_norm_bwd(dy, r, w, rs, d1, gate=gate)
    M.moe_post_norm_bwd(a, r, w, rs, a, gate=gate)
    assert torch.equal(a, d1)


def test_the_same_bits_every_time_and_in_a_graph(M):
    T, d = 700, 2880
    x, w, dy, gate = rand(T, d), rand(d, seed=1), rand(T, d, seed=2), rand(T, d, seed=3)
    rstd = full(T, t=F32)
    M.moe_norm_fwd(x, w, full(T, d), rstd, EPS)
    ws = torch.empty(M.moe_norm_workspace_bytes(T, d), dtype=torch.uint8, device="cuda")
    dx, dw, dg = full(T, d), full(d, t=F32), full(T, d)
    run = lambda: M.moe_post_norm_bwd(dy, x, w, rstd, dx, dw, ws, gate=gate, dgate=dg, gate_act=M.MOE_GATE_SIGMOID)  # noqa: E731
    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for rep in range(3):
        dy.copy_(rand(T, d, seed=10 + rep))
        run()
        want = [t.clone() for t in (dx, dw, dg)]
        for t in (dx, dw, dg):
            t.fill_(float("nan"))
        ws.fill_(255)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (dx, dw, dg))), rep


@pytest.mark.parametrize("cols", [1, "d"])
def test_gates_far_from_zero(M, cols):
    """A sigmoid's tails: its slope is e / (1 + e)^2 with e = exp(-|g|), whose argument's rounding costs |g| 2^-24 of it; what
    lies below fp32's normal range, 2^-126, may be 0."""
    far = [-float("inf"), -100.0, -85.0, -40.0, -17.0, -9.0, 0.0, 9.0, 17.0, 40.0, 85.0, 100.0, float("inf")]
    T, d = len(far), 512
    cols = d if cols == "d" else cols
    y, x, w, do = rand(T, d), torch.zeros(T, d, dtype=BF, device="cuda"), rand(d, std=0.3, mean=1.0, seed=2), rand(T, d, seed=3)
    gate = torch.tensor(far, dtype=BF, device="cuda").view(T, 1).expand(T, cols).contiguous()
    out, rstd = full(T, d), full(T, t=F32)
    M.moe_post_norm_fwd(y, x, w, out, rstd, EPS, gate=gate, gate_act=M.MOE_GATE_SIGMOID)
    yv, wv, dv, gv = bf16_values(y), bf16_values(w), bf16_values(do), bf16_values(gate)
    v = B.norm(yv, wv, EPS)[0]
    e = np.exp(-np.abs(gv))
    value, slope = np.where(gv < 0, e, 1.0) / (1 + e), e / (1 + e)**2
    arg = np.where(np.isfinite(gv), np.abs(gv), 0.0) * 2.0**-23 + 8 * 2.0**-24
    close(out, v * value, (HALF + SUM + arg) * np.abs(v * value) + 2.0**-125 * np.abs(v), "out")
    dy, dgate = full(T, d), full(T, cols, t=F32 if cols == 1 else BF)
    M.moe_post_norm_bwd(do, y, w, rstd, dy, gate=gate, dgate=dgate, gate_act=M.MOE_GATE_SIGMOID)
    if cols == 1:
        close(dgate, (dv * v).sum(1, keepdims=True) * slope,
              (2 * SUM + arg) * np.abs(dv * v).sum(1, keepdims=True) * slope + 2.0**-125 * np.abs(dv * v).sum(1, keepdims=True), "dgate")
    else:
        close(dgate, dv * v * slope, (HALF + SUM + arg) * np.abs(dv * v * slope) + 2.0**-125 * (1 + np.abs(dv * v)), "dgate")
    assert not dy.isnan().any()
