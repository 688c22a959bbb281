"""Router losses and their gradient against the fp64 oracle (GPU).

Bounds: a probability is exp(x - max) / sum: the exponent's argument is rounded once
(|x - max| 2^-24), exp and the reciprocal add a few 2^-23 and the sum of E terms at
most E 2^-24, so p is within P = (spread + E + 16) 2^-23 relative. Means over n tokens
of non-negative terms, summed in fp32, add n 2^-24 at most; the losses are sums of
non-negative terms of such factors. lse is off by at most P + |lse| 2^-23.
"""
import numpy as np
import pytest
import torch

from oracle import dense_oracle as D

pytestmark = pytest.mark.gpu
U = 2.0**-24


@pytest.fixture(scope="module")
def M():
    from ragged_grouped_gemm_device_amd import moe
    moe.load()
    return moe


def _run(M, lg, idx, valid=None, offs=None, cb=0.3, cz=0.02, grad=None, base=None, half=False):
    T, E = lg.shape
    S = 1 if offs is None else len(offs) - 1
    dev = "cuda"
    c = lambda a, t: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(t).cuda()  # noqa: E731
    g = dict(lg=c(lg, torch.float32), idx=c(idx, torch.int32), valid=c(valid, torch.uint8), seq=c(offs, torch.int32))
    out = dict(loss=torch.full((3,), float("nan"), device=dev), counts=torch.full((S, E), -7, dtype=torch.int32, device=dev),
               prob=torch.full((S, E), float("nan"), device=dev), tokens=torch.full((S + 2,), -7, dtype=torch.int32, device=dev))
    ws = torch.full((M.moe_balance_workspace_bytes(T, E, S),), 255, dtype=torch.uint8, device=dev)
    M.moe_balance_loss(g["lg"], g["idx"], out["loss"], out["counts"], out["prob"], out["tokens"], ws, cb, cz,
                       valid=g["valid"], seq_offsets=g["seq"])
    d = torch.full((T, E), float("nan"), device=dev) if base is None else c(base, torch.float32)
    d16 = torch.empty(T, E, dtype=torch.bfloat16, device=dev) if half else None
    up = None if grad is None else torch.tensor([grad], device=dev)
    M.moe_balance_loss_bwd(g["lg"], out["counts"], out["tokens"], d, idx.shape[1], cb, cz, valid=g["valid"],
                           seq_offsets=g["seq"], grad=up, accumulate=base is not None, dlogits_bf16=d16)
    torch.cuda.synchronize()
    got = {k: v.cpu().numpy() for k, v in out.items()}
    got["dlogits"] = d.cpu().numpy()
    if half:
        assert torch.equal(d16, d.to(torch.bfloat16))
    return got


def _check(got, lg, idx, valid=None, offs=None, cb=0.3, cz=0.02, grad=1.0, base=None):
    ref = D.balance_loss(lg, idx, valid, offs, cb, cz)
    T, E = lg.shape
    assert np.array_equal(got["counts"], ref["counts"])
    assert np.array_equal(got["tokens"], ref["tokens"])
    fin = lg[np.isfinite(lg)]
    spread = float(fin.max() - fin.min()) if fin.size else 0.0
    big = float(np.abs(fin).max()) if fin.size else 0.0
    P = (spread + E + 16) * 2 * U
    n = int(ref["tokens"][:-2].max())
    rel = P + (n + 8) * U
    assert (np.abs(got["prob"] - ref["prob"]) <= rel * ref["prob"] + 2.0**-120).all()
    lse = P + (big + np.log(E) + 1) * 2 * U     # absolute error of lse
    zrel = 2 * lse * np.sqrt(ref["loss"][2]) + lse * lse + (T + 8) * U * ref["loss"][2]
    brel = (rel + (E + 8) * U) * ref["loss"][1]
    assert abs(got["loss"][1] - ref["loss"][1]) <= brel
    assert abs(got["loss"][2] - ref["loss"][2]) <= zrel
    assert abs(got["loss"][0] - ref["loss"][0]) <= cb * brel + cz * zrel + 2 * U * ref["loss"][0]
    # gradient: p within P, f - f_ref exact to a few 2^-24 of the largest f, their mean within P of it
    nl, nt = max(int(ref["tokens"][-2]), 1), max(int(ref["tokens"][-1]), 1)
    k = idx.shape[1]
    seq = np.zeros(T, int)
    if offs is not None:
        seq = np.clip(np.searchsorted(offs, np.arange(T), side="right") - 1, 0, len(offs) - 2)
    ns = np.maximum(ref["tokens"][seq], 1)
    fmax = (ref["counts"].max(1) * E)[seq] / (k * ns)
    l64 = np.where(np.isfinite(lg), lg, -np.inf).astype(np.float64)
    mx = l64.max(1, keepdims=True)
    p = np.exp(l64 - np.where(np.isfinite(mx), mx, 0.0))     # 0 where no logit is finite
    p = p / np.maximum(p.sum(1, keepdims=True), 1e-300)
    bound = p * (cb / (nl * ns) * fmax * (2 * P + (E + 16) * U) + cz * 2 / nt * (lse + (big + np.log(E)) * (P + 8 * U)))[:, None]
    want = ref["dlogits"] * grad + (0 if base is None else base)
    bound = bound * abs(grad) * 2 + 2 * U * np.abs(want) + 2.0**-140
    assert (np.abs(got["dlogits"] - want) <= bound).all()


def _case(T, E, k, seed, scale=1.0):
    rng = np.random.default_rng(seed)
    lg = (rng.standard_normal((T, E)) * scale).astype(np.float32)
    return rng, lg, np.argsort(-lg, 1, kind="stable")[:, :k].astype(np.int32)


@pytest.mark.parametrize("T, E, k", [(1, 1, 1), (1, 8, 2), (5, 3, 3), (63, 8, 1), (256, 8, 2), (300, 12, 4), (129, 16, 1),
                                     (1000, 31, 8), (500, 32, 8), (777, 33, 2), (400, 64, 6), (211, 100, 5), (512, 128, 8),
                                     (150, 256, 8), (97, 400, 3), (40, 1024, 8), (3, 1024, 1024), (5000, 32, 4)])
def test_one_sequence(M, T, E, k):
    _, lg, idx = _case(T, E, k, T + E)
    _check(_run(M, lg, idx, half=True), lg, idx)


@pytest.mark.parametrize("T, E, k, S", [(10, 4, 2, 10), (100, 8, 2, 7), (1000, 32, 8, 16), (700, 60, 4, 33), (2100, 256, 8, 9),
                                        (128, 64, 4, 128), (130, 8, 2, 64), (1, 5, 2, 1), (2, 300, 3, 2), (3000, 7, 1, 2999)])
def test_ragged_masked_sequences(M, T, E, k, S):
    rng, lg, idx = _case(T, E, k, T * S)
    offs = np.sort(rng.integers(0, T + 1, S + 1)).astype(np.int32)   # empty ones, and tokens outside all of them
    offs[S // 2] = offs[S // 2 + 1]
    valid = (rng.random(T) < 0.8).astype(np.uint8)
    valid[offs[0]:offs[1]] = 0                                       # a sequence whose mask leaves nothing
    _check(_run(M, lg, idx, valid, offs), lg, idx, valid, offs)
    base = rng.standard_normal((T, E)).astype(np.float32)
    got = _run(M, lg, idx, valid, offs, grad=-2.5, base=base, half=True)
    _check(got, lg, idx, valid, offs, grad=-2.5, base=base)


def test_non_finite_logits_and_rows_left_empty(M):
    rng, lg, idx = _case(200, 20, 4, 3)
    lg[rng.random(lg.shape) < 0.2] = -np.inf
    lg[3] = -np.inf
    lg[4] = np.nan
    lg[5, 2], lg[6, 7] = np.inf, np.nan
    lg[7] = np.finfo(np.float32).min
    lg[8, 1:] = np.finfo(np.float32).min
    idx[9] = [-1, 20, 3, 3]                                          # out of range twice, the same index twice
    keep = np.ones(200, np.uint8)
    keep[7:9] = 0
    with np.errstate(over="ignore"):
        _check(_run(M, lg, idx, keep), lg, idx, keep)
    got = _run(M, lg, idx)                                           # the lowest value as a mask: finite results
    assert np.isfinite(got["dlogits"]).all() and np.isfinite(got["prob"]).all()
    nothing = _run(M, lg, idx, np.zeros(200, np.uint8))
    assert (nothing["loss"] == 0).all() and (nothing["dlogits"] == 0).all() and (nothing["counts"] == 0).all()


def test_collapsed_routing_keeps_its_small_gradient(M):
    """One expert far ahead of the others: the gradient is tiny and must not drown in rounding
    (P above is (30 + 8 + 16) 2^-23 = 6.4e-6; p and the mean of f carry it once each)."""
    rng, lg, _ = _case(64, 8, 1, 5)
    lg[np.arange(64), np.arange(64) % 3] += 24.0
    idx = np.argsort(-lg, 1)[:, :1].astype(np.int32)
    got = _run(M, lg, idx, cz=0.0)
    ref = D.balance_loss(lg, idx, balance_coef=0.3, z_coef=0.0)["dlogits"]
    assert np.linalg.norm(got["dlogits"] - ref) <= 2e-5 * np.linalg.norm(ref)


def test_same_bits_and_counts_of_the_router(M):
    rng, lg, _ = _case(3000, 32, 4, 8)
    cap = M.moe_capacity_rows(3000, 4, 32)
    i32 = dict(dtype=torch.int32, device="cuda")
    idx, counts = torch.empty(3000, 4, **i32), torch.empty(32, **i32)
    M.moe_route_counts(torch.from_numpy(lg).cuda(), 4, idx, torch.empty(3000, 4, device="cuda"), counts,
                       torch.empty(33, **i32), torch.empty(12000, **i32), torch.empty(cap, **i32), cap,
                       torch.zeros(1, **i32),
                       torch.empty(M.moe_route_workspace_bytes(3000, 4, 32), dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    a, b = (_run(M, lg, idx.cpu().numpy()) for _ in range(2))
    assert np.array_equal(a["counts"][0], counts.cpu().numpy())
    for key in a:
        assert np.array_equal(a[key], b[key]), key


def test_one_sequence_inside_the_batch_and_rows_off_16_bytes(M):
    """S = 1 with offsets (tokens before and behind it get gradient 0), and logits and gradients
    that start 4 bytes past a 16-byte boundary (element loads instead of 16-byte pieces)."""
    _, lg, idx = _case(120, 16, 3, 9)
    offs = np.array([17, 101], np.int32)
    _check(_run(M, lg, idx, offs=offs), lg, idx, offs=offs)
    T, E = lg.shape
    want = _run(M, lg, idx)
    hold = torch.empty(T * E + 1, device="cuda")
    off = hold[1:].view(T, E)
    off.copy_(torch.from_numpy(lg))
    g = torch.empty(T * E + 1, device="cuda")[1:].view(T, E)
    i32 = dict(dtype=torch.int32, device="cuda")
    loss, counts, prob, tokens = torch.empty(3, device="cuda"), torch.empty(1, E, **i32), torch.empty(1, E, device="cuda"), torch.empty(3, **i32)
    ws = torch.empty(M.moe_balance_workspace_bytes(T, E, 1), dtype=torch.uint8, device="cuda")
    M.moe_balance_loss(off, torch.from_numpy(idx).cuda(), loss, counts, prob, tokens, ws, 0.3, 0.02)
    M.moe_balance_loss_bwd(off, counts, tokens, g, 3, 0.3, 0.02)
    torch.cuda.synchronize()
    # another lane takes each expert, so the sums' order may differ: P above, 26 2^-23 + n 2^-24
    assert np.abs(g.cpu().numpy() - want["dlogits"]).max() <= 1e-4 * np.abs(want["dlogits"]).max()
    assert np.abs(loss.cpu().numpy() - want["loss"]).max() <= 3e-5 * want["loss"].max()
    assert np.array_equal(counts.cpu().numpy(), want["counts"])


def test_a_term_switched_off_stays_out(M):
    """A row of the type's lowest value: its squared log-sum-exp passes fp32, but with z_coef = 0 the
    loss is the balance loss alone, and the gradient finite."""
    _, lg, idx = _case(64, 8, 2, 6)
    lg[5] = np.finfo(np.float32).min
    for T in (64, 5000):
        x, i = np.resize(lg, (T, 8)), np.resize(idx, (T, 2))
        got = _run(M, x, i, cz=0.0)
        assert np.isinf(got["loss"][2]) and np.isfinite(got["dlogits"]).all()
        # fp32(0.3) and the stored loss[1] are each off by 2^-24 of themselves, as is the product
        assert abs(got["loss"][0] - 0.3 * got["loss"][1]) <= 3.1 * U * 0.3 * got["loss"][1]
