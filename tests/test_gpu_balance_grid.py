"""Router losses of more sequences than one launch has room for workgroups of (GPU)."""
import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0**-24


def test_more_sequences_than_a_launch_has_workgroups():
    """One token a sequence, 2^24 + 5 of them: joined by one workgroup each they would be 2^32 threads
    and more, past what a launch holds. With n_s = 1: f = 2 for the expert that is asked for, P = p, so
    B = mean of 2 p_chosen and Z = mean of lse^2. p is within P = (spread + 38) 2^-23 of itself, lse
    within L = P + (|lse| + 1) 2^-23; the last join is 64-bit."""
    from ragged_grouped_gemm_device_amd import moe as M
    T = (1 << 24) + 5
    g = torch.Generator("cuda").manual_seed(4)
    lg = torch.randn(T, 2, device="cuda", generator=g)
    idx = lg.argmax(1, keepdim=True).to(torch.int32)
    seq = torch.arange(T + 1, dtype=torch.int32, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    loss, counts, prob = torch.full((3,), float("nan"), device="cuda"), torch.full((T, 2), -7, **i32), torch.full((T, 2), -1.0, device="cuda")
    tokens = torch.full((T + 2,), -7, **i32)
    ws = torch.empty(M.moe_balance_workspace_bytes(T, 2, T), dtype=torch.uint8, device="cuda")
    M.moe_balance_loss(lg, idx, loss, counts, prob, tokens, ws, 0.3, 0.02, seq_offsets=seq)
    d = torch.full((T, 2), float("nan"), device="cuda")
    M.moe_balance_loss_bwd(lg, counts, tokens, d, 1, 0.3, 0.02, seq_offsets=seq)
    torch.cuda.synchronize()
    x = lg.double()
    p, lse = torch.softmax(x, 1), torch.logsumexp(x, 1)
    chosen = torch.zeros_like(counts).scatter_(1, idx.long(), 1)
    assert torch.equal(counts, chosen)
    assert (tokens[:T] == 1).all() and tokens[T:].tolist() == [T, T]
    spread, big = float((x[:, 0] - x[:, 1]).abs().max()), float(lse.abs().max())
    P = (spread + 38) * 2 * U
    L = P + (big + 1) * 2 * U
    assert ((prob.double() - p).abs() <= (P + 8 * U) * p).all()
    B, Z = float((2 * p * chosen).sum(1).mean()), float(lse.square().mean())
    zb = 2 * L * Z**0.5 + L * L + 8 * U * Z
    got = loss.tolist()
    assert abs(got[1] - B) <= (P + 16 * U) * B and abs(got[2] - Z) <= zb
    assert abs(got[0] - (0.3 * B + 0.02 * Z)) <= 0.3 * (P + 16 * U) * B + 0.02 * zb + 2 * U * got[0]
    f = 2.0 * chosen.double()
    want = 0.3 / T * p * (f - (p * f).sum(1, keepdim=True)) + 0.02 * 2 / T * lse.unsqueeze(1) * p
    bound = p * (0.3 / T * 2 * (2 * P + 54 * U) + 0.02 * 2 / T * (L + big * (P + 8 * U))) * 2 + 2 * U * want.abs() + 2.0**-140
    assert ((d.double() - want).abs() <= bound).all()
