"""Calls of the dense half at the edge of what its interface allows (GPU): outputs asked for one by one,
the largest widths, operands past 2^31 elements, tiles of more LDS stages than K has slabs.

References in 64 bits on the same bf16 inputs. Bounds: a sum of K products is off by at most (K + 2) 2^-24
of the sum of magnitudes, rounding to bf16 adds 2^-8; squared ReLU's slope is exact to 2^-23.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu
U, H = 2.0**-24, 2.0**-8
BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8


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


def _space(M, T, K, N):
    return torch.empty(max(16, M.moe_linear_workspace_bytes(T, K, N)), dtype=U8, device="cuda")


@pytest.mark.parametrize("T, N", [(1, 64), (7, 192), (300, 4096), (5000, 64)])
@pytest.mark.parametrize("act, z8", [(a, z) for a in ("swiglu", "srelu", "silu") for z in (False, True)] + [("none", False)])
def test_each_output_of_the_activation_backward_alone(M, T, N, act, z8):
    """dz, a and dbias are the same bits whether asked for alone or together."""
    new = _normal(T + N)
    code = {"swiglu": 0, "srelu": 2, "silu": 4, "none": 3}[act]
    NO = N // 2 if act == "swiglu" else N
    dy, z = new(T, NO), new(T, N)
    kw = dict(z=z)
    if act == "none":
        kw = {}
    elif z8:
        q, s = torch.empty(T, N, dtype=U8, device="cuda"), torch.empty(T, N // 32, dtype=U8, device="cuda")
        M.moe_quant_mxfp8(z, M.MOE_QUANT_ROWWISE, q, s)
        kw = dict(z_q=q, z_s=s)
    ws = _space(M, T, 8, N)
    outs = lambda: (torch.full((T, N), float("nan"), dtype=BF, device="cuda"),  # noqa: E731
                    None if act == "none" else torch.full((T, NO), float("nan"), dtype=BF, device="cuda"),
                    torch.full((N,), float("nan"), device="cuda"))
    dz, a, db = outs()
    M.moe_act_bwd(dy, dz, code, a=a, dbias=db, workspace=ws, **kw)
    dz1, a1, db1 = outs()
    M.moe_act_bwd(dy, dz1, code, **kw)
    if a1 is not None:
        M.moe_act_bwd(None, None, code, a=a1, **kw)
    ws.fill_(255)
    M.moe_act_bwd(dy, None, code, dbias=db1, workspace=ws, **kw)
    torch.cuda.synchronize()
    assert torch.equal(dz, dz1) and torch.equal(db, db1) and (a is None or torch.equal(a, a1))
    assert torch.isfinite(dz).all() and torch.isfinite(db).all()


@pytest.mark.parametrize("T, K, N", [(5, 1 << 20, 64), (70, 1 << 20, 64), (3, 64, 1 << 20), (70, 64, 1 << 20), (200, 8, 1 << 20),
                                     (200, 1 << 20, 8)])
def test_largest_widths(M, T, K, N):
    print(f"widths T={T} K={K} N={N}", flush=True)
    new = _normal(T)
    x, w, dz = new(T, K), new(K, N, std=K**-0.5), new(T, N)
    ws = _space(M, T, K, N)
    y, dx, dw = torch.empty(T, N, dtype=BF, device="cuda"), torch.empty(T, K, dtype=BF, device="cuda"), torch.empty(K, N, device="cuda")
    M.moe_linear_fwd(x, w, y, workspace=ws)
    M.moe_linear_dgrad(dz, w, dx, workspace=ws)
    M.moe_linear_wgrad(x, dz, dw, workspace=ws)
    torch.cuda.synchronize()
    xd, wd, dd = x.double(), w.double(), dz.double()
    ref, b = xd @ wd, (K + 2) * U * (xd.abs() @ wd.abs())
    _close(y, ref, b + H * (ref.abs() + b), "y")
    ref, b = dd @ wd.t(), (N + 2) * U * (dd.abs() @ wd.abs().t())
    _close(dx, ref, b + H * (ref.abs() + b), "dx")
    ref, b = xd.t() @ dd, (T + 2) * U * (xd.abs().t() @ dd.abs())
    _close(dw, ref, b, "dw")


def _tall_product(a, b):
    """a^T b over many rows, in 64 bits, and that of the magnitudes."""
    ref = torch.zeros(a.shape[1], b.shape[1], dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(ref)
    for i in range(0, a.shape[0], 10000):
        p, q = a[i:i + 10000].double(), b[i:i + 10000].double()
        ref += p.t() @ q
        mag += p.abs().t() @ q.abs()
    return ref, mag


def test_gradients_of_operands_past_2_to_the_31_elements(M):
    T, K, N = 140000, 16384, 64                 # x and dx hold 2.3e9 values
    new = _normal(8)
    x, dz, w = new(T, K), new(T, N), new(K, N)
    ws = _space(M, T, K, N)
    dw = torch.empty(K, N, device="cuda")
    M.moe_linear_wgrad(x, dz, dw, workspace=ws)
    q, s = torch.empty(T, K, dtype=U8, device="cuda"), torch.empty(T, K // 32, dtype=U8, device="cuda")
    M.moe_quant_mxfp8(x, M.MOE_QUANT_ROWWISE, q, s)
    dw8 = torch.empty(K, N, device="cuda")
    M.moe_linear_wgrad(None, dz, dw8, x_q=q, x_s=s, workspace=ws)
    torch.cuda.synchronize()
    ref, mag = _tall_product(x, dz)
    _close(dw, ref, (T + 2) * U * mag, "dw")
    M.moe_dequant_mxfp8(q, s, x)
    torch.cuda.synchronize()
    ref, mag = _tall_product(x, dz)
    _close(dw8, ref, (T + 2) * U * mag, "dw from the checkpoint")
    M.moe_linear_dgrad(dz, w, x, workspace=ws)
    torch.cuda.synchronize()
    wd = w.double()
    for r in (0, 131071, 131072, T - 1):
        dd = dz[r:r + 1].double()
        ref, b = dd @ wd.t(), (N + 2) * U * (dd.abs() @ wd.abs().t())
        _close(x[r:r + 1], ref, b + H * (ref.abs() + b), f"dx row {r}")
    # a reduction over the wide operand's columns
    wt, y = new(K, N), torch.empty(T, N, dtype=BF, device="cuda")
    M.moe_linear_fwd(x, wt, y, workspace=ws)
    torch.cuda.synchronize()
    for r in (0, 131072, T - 1):
        xd = x[r:r + 1].double()
        ref, b = xd @ wt.double(), (K + 2) * U * (xd.abs() @ wt.double().abs())
        _close(y[r:r + 1], ref, b + H * (ref.abs() + b), f"y row {r}")


@pytest.mark.parametrize("T, K, N", [(16401, 8, 72), (16890, 8, 136), (17180, 72, 8), (17070, 136, 8), (68, 3352, 272), (130, 4384, 208)])
def test_fewer_slabs_than_lds_stages(M, T, K, N):
    """128 x 128 tiles with four stages where K has two or three slabs of 64 (dgrad, forward, wgrad)."""
    new = _normal(N)
    x, w, dz = new(T, K), new(K, N), new(T, N)
    ws = _space(M, T, K, N)
    y, dx, dw = torch.full((T, N), float("nan"), dtype=BF, device="cuda"), torch.empty(T, K, dtype=BF, device="cuda"), torch.empty(K, N, device="cuda")
    M.moe_linear_fwd(x, w, y, workspace=ws)
    M.moe_linear_dgrad(dz, w, dx, workspace=ws)
    M.moe_linear_wgrad(x, dz, dw, workspace=ws)
    torch.cuda.synchronize()
    xd, wd, dd = x.double(), w.double(), dz.double()
    ref, b = xd @ wd, (K + 2) * U * (xd.abs() @ wd.abs())
    _close(y, ref, b + H * (ref.abs() + b), "y")
    ref, b = dd @ wd.t(), (N + 2) * U * (dd.abs() @ wd.abs().t())
    _close(dx, ref, b + H * (ref.abs() + b), "dx")
    ref, b = xd.t() @ dd, (T + 2) * U * (xd.abs().t() @ dd.abs())
    _close(dw, ref, b, "dw")
