"""The dense linear layer and its backward against the fp64 oracle (GPU).

Bounds, elementwise, from the arithmetic: a sum of K products of bf16 values (each
exact in fp32) accumulated in fp32 is off by at most K 2^-24 sum|x||w| in any order;
rounding the result to bf16 adds half a step, finfo(bf16).eps / 2 = 2^-8 of it. The
activations' own error: e^-x from the hardware's base-2 exponential of x log2(e)
rounded to fp32 is off by at most (2 |x| + 2) 2^-23 relative, and a reciprocal, erf
and products add a few 2^-23, so f and f' are within FN(x) = (2 |x| + 8) 2^-23 times
their largest possible size (|x| for f, 1.2 for f').
"""
import numpy as np
import pytest
import torch

from oracle import dense_oracle as D
from oracle import moe_oracle as O

from ._util import bf16_values

pytestmark = pytest.mark.gpu
U, H = 2.0**-24, 2.0**-8
BF = torch.bfloat16


@pytest.fixture(scope="module")
def M():
    from ragged_grouped_gemm_device_amd import moe
    moe.load()
    return moe


def _normal(rng, *shape, std=1.0):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32) * std).to(BF).cuda()


def _space(M, T, K, N):
    return torch.empty(max(16, M.moe_linear_workspace_bytes(T, K, N)), dtype=torch.uint8, device="cuda")


def _fn(v):
    return (2 * np.abs(v) + 8) * 2.0**-23


def _act_error(z, dzb, act):
    """Bound on |f(z + e) - f(z)| + the evaluation's own error for |e| <= dzb."""
    if act == "none":
        return dzb
    if act == "srelu":
        return (2 * np.abs(z) + dzb) * dzb + z * z * 2 * U
    if act in D.GATED:
        (g, u), (dg, du) = O.deinterleave(z), O.deinterleave(dzb)
        f = np.abs(D._f(g, act))
        df = 1.2 * dg + _fn(g) * np.abs(g)
        return df * (np.abs(u) + du) + f * du + f * np.abs(u) * 2 * U
    return 1.2 * dzb + _fn(z) * np.abs(z)


def _within(got, ref, bound, what):
    got, ref = np.asarray(got, np.float64), np.asarray(ref)
    assert got.shape == ref.shape
    bad = ~(np.abs(got - ref) <= bound + 2.0**-120)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3].tolist(), got[bad][:3], ref[bad][:3])


SHAPES = [  # one row; one chunk; odd rows and columns; K and N ending inside a slab and a tile
    (1, 8, 64), (1, 64, 64), (3, 72, 192), (31, 200, 128), (33, 2048, 256), (64, 1032, 64), (65, 64, 320),
    (127, 136, 192), (129, 328, 128), (300, 4096, 64), (1000, 328, 192), (257, 520, 576),
    (3001, 136, 4160),  # enough 256 x 256 tiles for the large tile
]


@pytest.mark.parametrize("T, K, N", SHAPES)
@pytest.mark.parametrize("act", D.ACTS)
def test_forward(M, T, K, N, act):
    print(f"forward T={T} K={K} N={N} act={act}", flush=True)
    rng = np.random.default_rng(T * 7 + K + N)
    x, w, b = _normal(rng, T, K), _normal(rng, K, N, std=K**-0.5), _normal(rng, N)
    NO = N // 2 if act in D.GATED else N
    r = _normal(rng, T, NO)
    xv, wv = bf16_values(x), bf16_values(w)
    ws = _space(M, T, K, N)
    code = D.ACTS.index(act)
    y0, z0 = D.linear(xv, wv, act, bf16_values(b), bf16_values(r))
    zb = (K + 2) * U * (np.abs(xv) @ np.abs(wv) + np.abs(bf16_values(b)))
    yb = _act_error(z0, zb, act)
    yb = yb + U * (np.abs(y0) + np.abs(bf16_values(r)))
    y = torch.full((T, NO), float("nan"), dtype=BF, device="cuda")
    y32 = torch.full((T, NO), float("nan"), device="cuda")
    M.moe_linear_fwd(x, w, y32, code, b, r, workspace=ws)
    if act == "none":
        M.moe_linear_fwd(x, w, y, code, b, r, workspace=ws)
        torch.cuda.synchronize()
    else:
        z = torch.full((T, N), float("nan"), dtype=BF, device="cuda")
        zq, zs = torch.full((T, N), 255, dtype=torch.uint8, device="cuda"), torch.zeros(T, N // 32, dtype=torch.uint8, device="cuda")
        M.moe_linear_fwd(x, w, y, code, b, r, z=z, z_q=zq, z_s=zs, workspace=ws)
        torch.cuda.synchronize()
        zv = bf16_values(z)
        _within(zv, z0, zb + H * (np.abs(z0) + zb), "z")
        q, s, _, _ = O.quant_mxfp8(zv, colwise=False)   # the checkpoint is that of the bf16 z, bit for bit
        assert np.array_equal(zq.cpu().numpy(), q) and np.array_equal(zs.cpu().numpy(), s)
    _within(y32.cpu().numpy(), y0, yb + U * np.abs(y0), "y fp32")
    _within(bf16_values(y), y0, yb + H * (np.abs(y0) + yb), "y")
    # without bias, residual and checkpoint; and the same bits when run again
    ya, yc = torch.empty_like(y), torch.empty_like(y)
    M.moe_linear_fwd(x, w, ya, code, workspace=ws)
    ws.fill_(255)
    M.moe_linear_fwd(x, w, yc, code, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(ya, yc)
    y1, z1 = D.linear(xv, wv, act)
    yb = _act_error(z1, (K + 2) * U * (np.abs(xv) @ np.abs(wv)), act)
    _within(bf16_values(ya), y1, yb + H * (np.abs(y1) + yb), "plain y")


@pytest.mark.parametrize("T, K, N", [(1, 8, 8), (5, 64, 24), (130, 72, 40), (40, 4096, 104)])
@pytest.mark.parametrize("act", ["none", "silu", "srelu"])
def test_forward_columns_off_the_block_grid(M, T, K, N, act):
    rng = np.random.default_rng(T + N)
    x, w = _normal(rng, T, K), _normal(rng, K, N, std=K**-0.5)
    y = torch.full((T + 1, N), 7.0, dtype=BF, device="cuda")
    M.moe_linear_fwd(x, w, y[:T], D.ACTS.index(act), workspace=_space(M, T, K, N))
    torch.cuda.synchronize()
    xv, wv = bf16_values(x), bf16_values(w)
    y0, z0 = D.linear(xv, wv, act)
    yb = _act_error(z0, (K + 2) * U * (np.abs(xv) @ np.abs(wv)), act)
    _within(bf16_values(y[:T]), y0, yb + H * (np.abs(y0) + yb), "y")
    assert (y[T] == 7.0).all()                     # nothing behind the last row


@pytest.mark.parametrize("T, K, N", SHAPES)
@pytest.mark.parametrize("act", D.ACTS)
@pytest.mark.parametrize("z8", [False, True])
def test_act_backward(M, T, K, N, act, z8):
    if act == "none" and z8:
        pytest.skip("nothing is kept without an activation")
    print(f"act_bwd T={T} N={N} act={act} z8={z8}", flush=True)
    rng = np.random.default_rng(T + N)
    NO = N // 2 if act in D.GATED else N
    dy, z = _normal(rng, T, NO), _normal(rng, T, N, std=2.0)
    ws = _space(M, T, K, N)
    kw = {}
    if z8:
        zq, zs = torch.empty(T, N, dtype=torch.uint8, device="cuda"), torch.empty(T, N // 32, dtype=torch.uint8, device="cuda")
        M.moe_quant_mxfp8(z, M.MOE_QUANT_ROWWISE, zq, zs)
        kw = dict(z_q=zq, z_s=zs)
        torch.cuda.synchronize()
        zv = O.mx_dequant(zq.cpu().numpy(), zs.cpu().numpy())
    else:
        zv = bf16_values(z)
        kw = {} if act == "none" else dict(z=z)
    dv = bf16_values(dy)
    dz = torch.full((T, N), float("nan"), dtype=BF, device="cuda")
    a = None if act == "none" else torch.full((T, NO), float("nan"), dtype=BF, device="cuda")
    db = torch.full((N,), float("nan"), device="cuda")
    M.moe_act_bwd(dy, dz, D.ACTS.index(act), a=a, dbias=db, workspace=ws, **kw)
    torch.cuda.synchronize()
    ref = D.act_backward(dv, zv, act)
    if act in D.GATED:
        g, u = O.deinterleave(zv)
        e = O.interleave(np.abs(dv * u) * 1.2 * _fn(g), np.abs(dv * g) * _fn(g))
    elif act in ("none", "srelu"):
        e = np.abs(ref) * 4 * U
    else:
        e = np.abs(dv) * 1.2 * _fn(zv)
    e = e + 4 * U * np.abs(ref)
    _within(bf16_values(dz), ref, e + H * (np.abs(ref) + e), "dz")
    _within(db.cpu().numpy(), ref.sum(0), e.sum(0) + (T + 2) * U * (np.abs(ref) + e).sum(0), "dbias")
    if a is not None:
        a0 = D.act_forward(zv, act)
        ab = _act_error(zv, np.zeros_like(zv), act)
        _within(bf16_values(a), a0, ab + H * (np.abs(a0) + ab), "a")
        a2 = torch.empty_like(a)                   # recomputation alone, no upstream gradient
        M.moe_act_bwd(None, None, D.ACTS.index(act), a=a2, **kw)
        torch.cuda.synchronize()
        assert torch.equal(a, a2)


@pytest.mark.parametrize("T, K, N", SHAPES + [(4100, 320, 136), (70, 64, 4096), (3000, 4104, 64), (20, 4168, 4104)])
def test_gradient_products(M, T, K, N):
    print(f"products T={T} K={K} N={N}", flush=True)
    rng = np.random.default_rng(T + K)
    x, w, dz, r = _normal(rng, T, K), _normal(rng, K, N, std=N**-0.5), _normal(rng, T, N), _normal(rng, T, K)
    ws = _space(M, T, K, N)
    xv, wv, dv, rv = (bf16_values(t) for t in (x, w, dz, r))
    dx = torch.full((T, K), float("nan"), dtype=BF, device="cuda")
    M.moe_linear_dgrad(dz, w, dx, workspace=ws)
    into = r.clone()
    M.moe_linear_dgrad(dz, w, into, residual=into, workspace=ws)   # added to the gradient that is there
    torch.cuda.synchronize()
    ref, b = dv @ wv.T, (N + 2) * U * (np.abs(dv) @ np.abs(wv).T)
    _within(bf16_values(dx), ref, b + H * (np.abs(ref) + b), "dx")
    b = b + 2 * U * np.abs(rv)
    _within(bf16_values(into), ref + rv, b + H * (np.abs(ref + rv) + b), "dx + r")

    ref, b = xv.T @ dv, (T + 2) * U * (np.abs(xv).T @ np.abs(dv))
    dw = torch.full((K, N), float("nan"), device="cuda")
    M.moe_linear_wgrad(x, dz, dw, workspace=ws)
    dwb = torch.full((K, N), float("nan"), dtype=BF, device="cuda")
    M.moe_linear_wgrad(x, dz, dwb, workspace=ws)
    torch.cuda.synchronize()
    _within(dw.cpu().numpy(), ref, b, "dw")
    _within(bf16_values(dwb), ref, b + H * (np.abs(ref) + b), "dw bf16")
    first = dw.clone()
    M.moe_linear_wgrad(x, dz, dw, accumulate=True, workspace=ws)
    torch.cuda.synchronize()
    _within(dw.cpu().numpy(), first.cpu().numpy().astype(np.float64) + ref, b + 2 * U * (2 * np.abs(ref) + b), "dw accumulated")
    if K % 32 == 0:
        xq, xs = torch.empty(T, K, dtype=torch.uint8, device="cuda"), torch.empty(T, K // 32, dtype=torch.uint8, device="cuda")
        M.moe_quant_mxfp8(x, M.MOE_QUANT_ROWWISE, xq, xs)
        M.moe_linear_wgrad(None, dz, dw, x_q=xq, x_s=xs, workspace=ws)
        torch.cuda.synchronize()
        x8 = O.mx_dequant(xq.cpu().numpy(), xs.cpu().numpy())
        ref, b = x8.T @ dv, (T + 2) * U * (np.abs(x8).T @ np.abs(dv))
        _within(dw.cpu().numpy(), ref, b, "dw from the checkpoint")


def test_dequant_every_code_and_scale(M):
    codes = np.tile(np.arange(256, dtype=np.uint8), (256, 1))
    scales = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 8, 1)
    out = torch.empty(256, 256, dtype=BF, device="cuda")
    M.moe_dequant_mxfp8(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), out)
    torch.cuda.synchronize()
    got = bf16_values(out)
    ref = O.round_bf16(O.mx_dequant(codes, np.minimum(scales, 254)))   # past bf16's range: infinite
    ref[255] = np.nan
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    ok = ~np.isnan(ref)
    assert np.array_equal(got[ok], ref[ok])
    assert np.array_equal(np.signbit(got[ok]), np.signbit(ref[ok]))


@pytest.mark.parametrize("R, C", [(1, 32), (3, 96), (1021, 2880), (257, 4096)])
def test_dequant_restores_the_quantizer(M, R, C):
    x = _normal(np.random.default_rng(R), R, C, std=3.0)
    q, s = torch.empty(R, C, dtype=torch.uint8, device="cuda"), torch.empty(R, C // 32, dtype=torch.uint8, device="cuda")
    M.moe_quant_mxfp8(x, M.MOE_QUANT_ROWWISE, q, s)
    out = torch.full((R + 1, C), 7.0, dtype=BF, device="cuda")
    M.moe_dequant_mxfp8(q, s, out[:R])
    torch.cuda.synchronize()
    assert np.array_equal(bf16_values(out[:R]), O.mx_dequant(q.cpu().numpy(), s.cpu().numpy()))
    assert (out[R] == 7.0).all()


def test_other_stream_device_and_refusals(M):
    x, w, y = torch.zeros(4, 64, dtype=BF, device="cuda"), torch.zeros(64, 128, dtype=BF, device="cuda"), torch.zeros(4, 128, dtype=BF)
    with pytest.raises(ValueError):
        M.moe_linear_fwd(x, w, y)                       # y is on the host
    with pytest.raises(M.MoEError):
        M.moe_linear_fwd(torch.zeros(1, 8192, dtype=BF, device="cuda"), torch.zeros(8192, 128, dtype=BF, device="cuda"),
                         torch.zeros(1, 128, dtype=BF, device="cuda"))   # split product without a workspace
    rng = np.random.default_rng(0)
    x, w = _normal(rng, 48, 1024), _normal(rng, 1024, 256)
    y0, y1 = torch.empty(48, 256, dtype=BF, device="cuda"), torch.empty(48, 256, dtype=BF, device="cuda")
    M.moe_linear_fwd(x, w, y0, workspace=_space(M, 48, 1024, 256))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        M.moe_linear_fwd(x, w, y1, workspace=_space(M, 48, 1024, 256))
    side.synchronize()
    assert torch.equal(y0, y1)


def test_infinities_and_nan_stay_in_their_rows_and_columns(M):
    """Nothing that lies past the end of K, of a tile or of the rows meets a non-finite value."""
    rng = np.random.default_rng(1)
    for T, K, N in ((5, 72, 64), (70, 200, 136), (300, 1096, 264), (3001, 136, 4160)):
        x, w, dz = _normal(rng, T, K), _normal(rng, K, N), _normal(rng, T, N)
        x[T - 1, K - 1], x[0, 3] = float("inf"), float("nan")
        w[K - 1, N - 1] = float("inf")
        ws = _space(M, T, K, N)
        y, dx, dw = torch.empty(T, N, dtype=BF, device="cuda"), torch.empty(T, K, dtype=BF, device="cuda"), torch.empty(K, N, device="cuda")
        M.moe_linear_fwd(x, w, y, workspace=ws)
        M.moe_linear_dgrad(dz, w, dx, workspace=ws)
        M.moe_linear_wgrad(x, dz, dw, workspace=ws)
        torch.cuda.synchronize()
        bad = ~torch.isfinite(y)
        assert bad[0].all() and bad[T - 1].all() and bad[:, N - 1].all()
        assert not bad[1:T - 1, :N - 1].any()
        bad = ~torch.isfinite(dx)
        assert bad[:, K - 1].all() and not bad[:, :K - 1].any()
        bad = ~torch.isfinite(dw)
        assert bad[3].all() and bad[K - 1].all()
        keep = torch.ones(K, dtype=torch.bool)
        keep[[3, K - 1]] = False
        assert not bad[keep.cuda()].any()


@pytest.mark.parametrize("T, K, N, stage", [(1, 8192, 4096, "f"), (48, 4096, 512, "f"), (200, 8192, 1024, "d"), (8192, 256, 256, "w"),
                                            (4300, 4104, 4168, "f"), (4300, 4104, 4168, "w")])
def test_captured_products_replay_to_the_eager_bits(M, T, K, N, stage):
    """Products whose K is split: the joined sums are the same in every replay, with other work between."""
    rng = np.random.default_rng(T)
    x, w, dz = _normal(rng, T, K), _normal(rng, K, N, std=0.02), _normal(rng, T, N)
    ws = _space(M, T, K, N)
    out = torch.empty({"f": (T, N), "d": (T, K), "w": (K, N)}[stage], dtype=BF, device="cuda")
    call = {"f": lambda: M.moe_linear_fwd(x, w, out, workspace=ws), "d": lambda: M.moe_linear_dgrad(dz, w, out, workspace=ws),
            "w": lambda: M.moe_linear_wgrad(x, dz, out, workspace=ws)}[stage]
    call()
    torch.cuda.synchronize()
    want = out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for _ in range(3):
        out.fill_(float("nan"))
        ws.fill_(255)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_large_offsets(M):
    """Rows and columns whose element offsets pass 2^31: the last rows of a tall input and output."""
    T, K, N = 140000, 16, 16384                 # y holds 2.3e9 values
    g = torch.Generator("cuda").manual_seed(2)
    x = torch.randn(T, K, device="cuda", generator=g).to(BF)
    w = torch.randn(K, N, device="cuda", generator=g).to(BF)
    y = torch.empty(T, N, dtype=BF, device="cuda")
    ws = _space(M, T, K, N)
    M.moe_linear_fwd(x, w, y, workspace=ws)
    torch.cuda.synchronize()
    wv = bf16_values(w)
    for r in (0, 131071, 131072, T - 1):
        xv = bf16_values(x[r:r + 1])
        ref, b = xv @ wv, (K + 2) * U * (np.abs(xv) @ np.abs(wv))
        _within(bf16_values(y[r:r + 1]), ref, b + H * (np.abs(ref) + b), f"row {r}")
    q, s = torch.empty(T, N, dtype=torch.uint8, device="cuda"), torch.empty(T, N // 32, dtype=torch.uint8, device="cuda")
    M.moe_quant_mxfp8(y, M.MOE_QUANT_ROWWISE, q, s)
    M.moe_dequant_mxfp8(q, s, y)
    torch.cuda.synchronize()
    assert np.array_equal(bf16_values(y[-2:]), O.mx_dequant(q[-2:].cpu().numpy(), s[-2:].cpu().numpy()))
    dy = torch.randn(T, N // 2, device="cuda", generator=g).to(BF)
    M.moe_act_bwd(dy, y, M.MOE_ACT_SWIGLU, z_q=q, z_s=s)
    torch.cuda.synchronize()
    zv = O.mx_dequant(q[-1:].cpu().numpy(), s[-1:].cpu().numpy())
    dv = bf16_values(dy[-1:])
    ref = D.act_backward(dv, zv, "swiglu")
    gt, up = O.deinterleave(zv)
    e = O.interleave(np.abs(dv * up) * 1.2 * _fn(gt), np.abs(dv * gt) * _fn(gt)) + 4 * U * np.abs(ref)
    _within(bf16_values(y[-1:]), ref, e + H * (np.abs(ref) + e), "dz")


def test_gelu_keeps_its_tail(M):
    """GELU in fp32 on exact arguments: relative precision far into the negative tail. exp's
    argument x^2 / 2 is rounded twice (2^-23 of it in all, times log2 e in the base-2 form);
    polynomial, reciprocal, exponential and products add less than 2^-19."""
    v = torch.linspace(-12.5, 12.5, 4001).to(BF).cuda()
    x = torch.zeros(4001, 8, dtype=BF, device="cuda")
    x[:, 0] = v
    w = torch.zeros(8, 64, dtype=BF, device="cuda")
    w[0] = 1.0
    y = torch.empty(4001, 64, device="cuda")
    M.moe_linear_fwd(x, w, y, M.MOE_ACT_GELU, workspace=_space(M, 4001, 8, 64))
    torch.cuda.synchronize()
    from scipy.special import ndtr
    vv = bf16_values(v)
    ref = vv * ndtr(vv)
    bound = np.abs(ref) * (2.0**-19 + vv * vv / 2 * 2.0**-22)
    _within(y[:, 0].cpu().numpy(), ref, bound, "gelu")
    _within(y[:, 63].cpu().numpy(), ref, bound, "gelu")


@pytest.mark.parametrize("T", [3, 300])
@pytest.mark.parametrize("act", ["swiglu", "geglu", "srelu", "silu", "gelu", "none"])
def test_a_nan_passes_every_activation(M, act, T):
    """NaN in a row of x reaches all of that row's y, z, dz and a, and no other row."""
    rng = np.random.default_rng(3)
    K, N = 72, 128
    code, NO = {"swiglu": 0, "geglu": 1, "srelu": 2, "none": 3, "silu": 4, "gelu": 5}[act], 64 if "glu" in act else 128
    x, w, dy = _normal(rng, T, K), _normal(rng, K, N), _normal(rng, T, NO)
    x[1, 7] = float("nan")
    ws = _space(M, T, K, N)
    y, z = torch.empty(T, NO, dtype=BF, device="cuda"), torch.empty(T, N, dtype=BF, device="cuda")
    keep = {} if act == "none" else {"z": z}
    M.moe_linear_fwd(x, w, y, code, workspace=ws, **keep)
    outs = [y]
    if act != "none":
        dz, a = torch.empty_like(z), torch.empty_like(y)
        M.moe_act_bwd(dy, dz, code, z=z, a=a)
        outs += [z, dz, a]
    torch.cuda.synchronize()
    for o in outs:
        bad = torch.isnan(o)
        assert bad[1].all() and int(bad.sum()) == o.shape[1], act
