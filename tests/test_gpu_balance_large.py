"""Router losses and their gradient where a workgroup passes several times over its tokens (GPU),
against the same formulas in 64-bit torch.

Bounds. A probability is exp(x - max) / sum: the exponent's argument is rounded once (|x - max| 2^-24);
exponential, reciprocal and product add a few 2^-23, and a lane adds at most 16 terms and the lanes
join in at most 6 steps, so p is within P = (spread + 38) 2^-23 of itself. A mean over tokens adds
non-negative terms: at most all tokens of a chunk one after the other (T / 1024 + 128), 128 chunks a
lane and 32 more joins, DEPTH 2^-24 of the sum. lse is off by at most L = P + (|lse| + 1) 2^-23.
"""
import random

import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0**-24
D = torch.float64


@pytest.fixture(scope="module")
def M():
    from ragged_grouped_gemm_device_amd import moe
    moe.load()
    return moe


def _inputs(T, E, k, S, seed, mask):
    g = torch.Generator("cuda").manual_seed(seed)
    lg = torch.randn(T, E, device="cuda", generator=g) * 1.5
    idx = lg.topk(k, 1).indices.to(torch.int32)
    seq = valid = None
    if S > 1:
        cuts = torch.randint(0, T + 1, (S - 1,), device="cuda", generator=g).sort().values
        seq = torch.cat((torch.tensor([min(3, T - 1)], device="cuda"), cuts.clamp(min=min(3, T - 1)),
                         torch.tensor([max(T - 2, min(3, T - 1))], device="cuda"))).sort().values.to(torch.int32)
    if mask:
        valid = (torch.rand(T, device="cuda", generator=g) < 0.9).to(torch.uint8)
        lg[torch.rand(lg.shape, device="cuda", generator=g) < 0.05] = float("-inf")
        lg[T // 2] = float("nan")
    return lg, idx, valid, seq


def _buffers(M, T, E, S):
    dev = dict(device="cuda")
    return (torch.full((3,), float("nan"), **dev), torch.full((S, E), -7, dtype=torch.int32, **dev),
            torch.full((S, E), float("nan"), **dev), torch.full((S + 2,), -7, dtype=torch.int32, **dev),
            torch.full((M.moe_balance_workspace_bytes(T, E, S),), 255, dtype=torch.uint8, **dev))


def _reference(lg, idx, valid, seq, cb, cz):
    """loss, counts, prob, tokens, and what the gradient's bound takes: dlogits, p, lse, n_s and f by token."""
    (T, E), k = lg.shape, idx.shape[1]
    S = 1 if seq is None else len(seq) - 1
    at = torch.arange(T, device="cuda")
    own = torch.zeros_like(at) if seq is None else torch.searchsorted(seq.long(), at, right=True) - 1
    inside = (own >= 0) & (own < S)
    x = torch.where(torch.isfinite(lg), lg.to(D), float("-inf"))
    live = inside & torch.isfinite(lg).any(1)
    if valid is not None:
        live &= valid != 0
    own = own.clamp(0, S - 1)
    top = torch.where(live, x.amax(1), 0.0)
    e = torch.where(live.unsqueeze(1), torch.exp(x - top.unsqueeze(1)), 0.0)
    tot = e.sum(1)
    p = e / torch.where(live, tot, 1.0).unsqueeze(1)
    lse = torch.where(live, top + torch.log(torch.where(live, tot, 1.0)), 0.0)
    n = torch.zeros(S, device="cuda", dtype=torch.int64).index_add_(0, own, live.long())
    counts = torch.zeros(S * E, device="cuda", dtype=torch.int64)
    counts.index_add_(0, (own.unsqueeze(1) * E + idx)[live].reshape(-1), torch.ones_like(idx, dtype=torch.int64)[live].reshape(-1))
    counts = counts.view(S, E)
    per = n.clamp(min=1).unsqueeze(1)
    prob = torch.zeros(S, E, device="cuda", dtype=D).index_add_(0, own, p) / per
    f = counts * E / (k * per).to(D)
    nl, nt = int((n > 0).sum()), int(n.sum())
    bal, z = (f * prob).sum() / max(nl, 1), lse.square().sum() / max(nt, 1)
    ft = f[own]
    w = 1.0 / (max(nl, 1) * per[own].to(D))
    d = cb * w * p * (ft - (p * ft).sum(1, keepdim=True)) + cz * 2 / max(nt, 1) * lse.unsqueeze(1) * p
    return dict(loss=(cb * bal + cz * z, bal, z), counts=counts, prob=prob, n=n, nl=nl, nt=nt, dlogits=d, p=p, lse=lse,
                w=w, fmax=ft.amax(1, keepdim=True))


def _check(M, lg, idx, valid, seq, cb=0.3, cz=0.02, up=None, base=None):
    (T, E), k = lg.shape, idx.shape[1]
    S = 1 if seq is None else len(seq) - 1
    loss, counts, prob, tokens, ws = _buffers(M, T, E, S)
    M.moe_balance_loss(lg, idx, loss, counts, prob, tokens, ws, cb, cz, valid=valid, seq_offsets=seq)
    d = torch.full((T, E), float("nan"), device="cuda") if base is None else base.clone()
    d16 = torch.empty(T, E, dtype=torch.bfloat16, device="cuda")
    grad = None if up is None else torch.tensor([up], device="cuda")
    M.moe_balance_loss_bwd(lg, counts, tokens, d, k, cb, cz, valid=valid, seq_offsets=seq, grad=grad,
                           accumulate=base is not None, dlogits_bf16=d16)
    torch.cuda.synchronize()
    r = _reference(lg, idx, valid, seq, cb, cz)
    assert torch.equal(counts.long(), r["counts"])
    assert torch.equal(tokens.long(), torch.cat((r["n"], torch.tensor([r["nl"], r["nt"]], device="cuda"))))
    fin = lg[torch.isfinite(lg)]
    spread = float(fin.max() - fin.min())
    P = (spread + 38) * 2 * U
    rel = P + (T / 1024 + 128 + 128 + 32) * U
    assert ((prob.to(D) - r["prob"]).abs() <= rel * r["prob"] + 2.0**-120).all()
    lerr = P + (float(r["lse"].abs().max()) + 1) * 2 * U
    zrel = 2 * lerr * float(r["loss"][2])**0.5 + lerr * lerr + rel * float(r["loss"][2])
    brel = (rel + 40 * U) * float(r["loss"][1])
    got = loss.tolist()
    assert abs(got[1] - float(r["loss"][1])) <= brel
    assert abs(got[2] - float(r["loss"][2])) <= zrel
    assert abs(got[0] - float(r["loss"][0])) <= cb * brel + cz * zrel + 2 * U * abs(float(r["loss"][0]))
    g = 1.0 if up is None else up
    want = r["dlogits"] * g + (0 if base is None else base.to(D))
    big = float(r["lse"].abs().max())
    bound = r["p"] * (cb * r["w"] * r["fmax"] * (2 * P + 54 * U) + cz * 2 / max(r["nt"], 1) * (lerr + big * (P + 8 * U)))
    bound = bound * abs(g) * 2 + 2 * U * want.abs() + 2.0**-140
    bad = ~((d.to(D) - want).abs() <= bound)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist())
    assert torch.equal(d16, d.to(torch.bfloat16))


# tokens a step: 128 with at most 16 experts, 64 with 32, 32 with 256, 16 with 512, 8 beyond; a chunk is
# about T / 1024 tokens forward and T / 2048 backward, so here both take two steps and more
@pytest.mark.parametrize("T, E, k, S, mask", [
    (300007, 8, 2, 1, False), (300001, 3, 1, 40, True), (600000, 16, 1, 300, True), (140000, 32, 8, 1, True),
    (140001, 31, 4, 5, False), (70001, 64, 6, 64, True), (70003, 127, 2, 9, False), (70001, 256, 8, 64, False),
    (131072, 256, 8, 64, True), (40000, 400, 3, 16, True), (33001, 511, 5, 1, False), (20000, 1024, 8, 1, True),
    (20003, 1023, 4, 37, True), (50000, 1000, 8, 3, False), (150000, 250, 1, 2, True)])
def test_several_passes_over_a_chunk(M, T, E, k, S, mask):
    print(f"losses T={T} E={E} k={k} S={S} mask={mask}", flush=True)
    lg, idx, valid, seq = _inputs(T, E, k, S, T + E, mask)
    _check(M, lg, idx, valid, seq)
    base = torch.randn(T, E, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    _check(M, lg, idx, valid, seq, up=-2.5, base=base)


@pytest.mark.parametrize("i", range(16))
def test_random_losses_and_probabilities(M, i):
    rng = random.Random(500 + i)
    E = rng.choice([rng.randint(1, 1024), 1 << rng.randint(0, 10)])
    T = min(int(400000 ** rng.random()) + 1, (1 << 25) // E)
    k, S = rng.randint(1, min(E, 8)), rng.randint(1, max(1, min(T, 200)))
    mask = rng.random() < 0.5
    print(f"losses {i}: T={T} E={E} k={k} S={S} mask={mask}", flush=True)
    _check(M, *_inputs(T, E, k, S, i, mask and T > 1))


def test_one_long_sequence_among_short_and_empty_ones(M):
    T, E = 120000, 24
    lg, idx, _, _ = _inputs(T, E, 2, 1, 5, False)
    ends = [0] * 7 + list(range(1, 60)) + [60] * 900 + [T - 40] + [T - 40] * 900 + list(range(T - 39, T + 1))
    _check(M, lg, idx, None, torch.tensor(ends, dtype=torch.int32, device="cuda"))


def test_captured_losses_replay_to_the_eager_bits(M):
    T, E, k, S = 70001, 256, 8, 64
    lg, idx, valid, seq = _inputs(T, E, k, S, 9, True)
    loss, counts, prob, tokens, ws = _buffers(M, T, E, S)
    d = torch.empty(T, E, device="cuda")

    def call():
        M.moe_balance_loss(lg, idx, loss, counts, prob, tokens, ws, 0.3, 0.02, valid=valid, seq_offsets=seq)
        M.moe_balance_loss_bwd(lg, counts, tokens, d, k, 0.3, 0.02, valid=valid, seq_offsets=seq)

    call()
    torch.cuda.synchronize()
    outs = (loss, counts, prob, tokens, d)
    want = [o.clone() for o in outs]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for _ in range(3):
        for o in outs:
            o.fill_(7)
        ws.fill_(255)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)
