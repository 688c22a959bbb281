"""Every form of the dense products that the plan can choose and the other tests' shapes do not reach:
tile, K in pieces, how the pieces are joined (GPU). tests/test_dense_plan.py holds the list against the
plan.

References in 64 bits on the same bf16 inputs. Bounds: a sum of K products is off by at most (K + 2) 2^-24
of the sum of magnitudes, rounding to bf16 adds 2^-8. An activation moves that by its slope, at most 1.2
for SiLU and GELU, and is itself within (2 |v| + 8) 2^-23 |v|: the exponential's argument is rounded
once, a reciprocal and a few products follow.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu
U, H = 2.0**-24, 2.0**-8
BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8

# T, K, N: those that every activation runs with, then those whose gradients are of interest, the last of
# which have so few outputs that eight lanes join an output's pieces
FORWARD = [(10959, 3360, 320), (14190, 7608, 320), (9, 1824, 4416), (9, 1056, 64), (21, 1312, 3136), (1, 1824, 4416),
           (131, 280, 5504), (3511, 880, 4736), (17913, 200, 192), (9, 208, 64)]
FORMS = FORWARD + [(1, 4448, 2624), (9, 4160, 1984), (9, 32, 1088), (1, 4160, 1920), (2187, 96, 2112), (7501, 160, 4160),
                   (4396, 32, 4416), (5597, 1648, 272), (1812, 192, 6280), (25424, 3064, 784), (2113, 4192, 8),
                   (2127, 8, 3768), (4421, 8, 8184), (4114, 2368, 8), (15953, 2168, 8), (1090, 4120, 8)]


@pytest.fixture(scope="module")
def M():
    from ragged_grouped_gemm_device_amd import moe
    moe.load()
    return moe


def _close(got, ref, bound, what):
    bad = ~((got.double() - ref).abs() <= bound + 2.0**-120)
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:3].tolist())


def _normal(seed):
    g = torch.Generator("cuda").manual_seed(seed)
    return lambda *s, std=1.0: (torch.randn(*s, device="cuda", generator=g) * std).to(BF)


def _space(M, T, K, N, passes):
    """A workspace of just the bytes asked for, with guard bytes behind it."""
    n = max(16, M.moe_linear_workspace_bytes(T, K, N, passes))
    whole = torch.full((n + 4096,), 77, dtype=U8, device="cuda")
    return whole[:n], whole[n:]


def _unary(v, e, name):
    """f(v) and the bound on its change for an error e of v."""
    if name == "none":
        return v, e
    if name == "srelu":
        return v.clamp(min=0).square(), (2 * v.abs() + e) * e + 4 * U * v * v
    f = v * torch.sigmoid(v) if name == "silu" else v * torch.special.ndtr(v)
    return f, 1.2 * e + (2 * v.abs() + 8) * 2 * U * v.abs()


ACTS = ("swiglu", "geglu", "srelu", "none", "silu", "gelu")


@pytest.mark.parametrize("T, K, N, act", [(*s, a) for s in FORWARD for a in ACTS] + [(*s, "none") for s in FORMS[len(FORWARD):]])
def test_forward_forms(M, T, K, N, act):
    gated = act in ("swiglu", "geglu")
    print(f"forward T={T} K={K} N={N} act={act}", flush=True)
    new = _normal(T + N)
    NO = N // 2 if gated else N
    x, w, b, r = new(T, K), new(K, N, std=K**-0.5), new(N), new(T, NO)
    code = {"swiglu": 0, "geglu": 1, "srelu": 2, "none": 3, "silu": 4, "gelu": 5}[act]
    ws, guard = _space(M, T, K, N, M.MOE_LINEAR_FWD)
    y, y32 = torch.full((T, NO), float("nan"), dtype=BF, device="cuda"), torch.full((T, NO), float("nan"), device="cuda")
    keep = {}
    if act != "none":
        keep = dict(z=torch.full((T, N), float("nan"), dtype=BF, device="cuda"), z_q=torch.full((T, N), 255, dtype=U8, device="cuda"),
                    z_s=torch.full((T, N // 32), 255, dtype=U8, device="cuda"))
    M.moe_linear_fwd(x, w, y, code, b, r, workspace=ws, **keep)
    ws.fill_(255)
    M.moe_linear_fwd(x, w, y32, code, b, workspace=ws)
    into = r.clone()                                        # the residual is the output itself
    ws.fill_(255)
    M.moe_linear_fwd(x, w, into, code, b, into, workspace=ws)
    torch.cuda.synchronize()
    assert (guard == 77).all()
    assert torch.equal(into, y)
    xd, wd, bd, rd = x.double(), w.double(), b.double(), r.double()
    z0 = xd @ wd + bd
    zb = (K + 2) * U * (xd.abs() @ wd.abs() + bd.abs())
    if keep:
        _close(keep["z"], z0, zb + H * (z0.abs() + zb), "z")
        q, s = torch.empty_like(keep["z_q"]), torch.empty_like(keep["z_s"])
        M.moe_quant_mxfp8(keep["z"], M.MOE_QUANT_ROWWISE, q, s)
        torch.cuda.synchronize()
        assert torch.equal(q, keep["z_q"]) and torch.equal(s, keep["z_s"])
    if gated:
        (g, u), (gb, ub) = ([v.reshape(T, -1, 2, 32)[:, :, j].reshape(T, -1) for j in (0, 1)] for v in (z0, zb))
        f, fb = _unary(g, gb, "silu" if act == "swiglu" else "gelu")
        ref, bound = f * u, fb * (u.abs() + ub) + f.abs() * ub + 4 * U * (f * u).abs()
    else:
        ref, bound = _unary(z0, zb, act)
    _close(y32, ref, bound + 2 * U * ref.abs(), "y fp32")
    ref, bound = ref + rd, bound + 2 * U * (ref.abs() + rd.abs())
    _close(y, ref, bound + H * (ref.abs() + bound), "y")


@pytest.mark.parametrize("T, K, N", FORMS)
def test_gradient_forms(M, T, K, N):
    print(f"gradients T={T} K={K} N={N}", flush=True)
    new = _normal(T + K)
    x, w, dz = new(T, K), new(K, N, std=N**-0.5), new(T, N)
    ws, guard = _space(M, T, K, N, M.MOE_LINEAR_BWD)
    dx, into = torch.full((T, K), float("nan"), dtype=BF, device="cuda"), x.clone()
    M.moe_linear_dgrad(dz, w, dx, workspace=ws)
    ws.fill_(255)
    M.moe_linear_dgrad(dz, w, into, residual=into, workspace=ws)
    dw, dwb = torch.full((K, N), float("nan"), device="cuda"), torch.full((K, N), float("nan"), dtype=BF, device="cuda")
    base = torch.randn(K, N, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    added = base.clone()
    for out, add in ((dw, False), (dwb, False), (added, True)):
        ws.fill_(255)
        M.moe_linear_wgrad(x, dz, out, accumulate=add, workspace=ws)
    torch.cuda.synchronize()
    assert (guard == 77).all()
    xd, wd, dd = x.double(), w.double(), dz.double()
    ref, b = dd @ wd.t(), (N + 2) * U * (dd.abs() @ wd.abs().t())
    _close(dx, ref, b + H * (ref.abs() + b), "dx")
    ref, b = ref + xd, b + 2 * U * (ref.abs() + xd.abs())
    _close(into, ref, b + H * (ref.abs() + b), "dx + r")
    ref, b = xd.t() @ dd, (T + 2) * U * (xd.abs().t() @ dd.abs())
    _close(dw, ref, b, "dw")
    _close(dwb, ref, b + H * (ref.abs() + b), "dw bf16")
    _close(added, ref + base.double(), b + 2 * U * (ref.abs() + base.double().abs()), "dw accumulated")
    if K % 32:
        return
    xq, xs, back = torch.empty(T, K, dtype=U8, device="cuda"), torch.empty(T, K // 32, dtype=U8, device="cuda"), torch.empty(T, K, dtype=BF, device="cuda")
    M.moe_quant_mxfp8(x, M.MOE_QUANT_ROWWISE, xq, xs)
    M.moe_dequant_mxfp8(xq, xs, back)
    added.copy_(base)
    for out, add in ((dw, False), (dwb, False), (added, True)):
        ws.fill_(255)
        M.moe_linear_wgrad(None, dz, out, x_q=xq, x_s=xs, accumulate=add, workspace=ws)
    torch.cuda.synchronize()
    assert (guard == 77).all()
    ref, b = back.double().t() @ dd, (T + 2) * U * (back.double().abs().t() @ dd.abs())
    _close(dw, ref, b, "dw from the checkpoint")
    _close(dwb, ref, b + H * (ref.abs() + b), "dw bf16 from the checkpoint")
    _close(added, ref + base.double(), b + 2 * U * (ref.abs() + base.double().abs()), "dw accumulated from the checkpoint")
