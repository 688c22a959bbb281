"""Experts served on 4-bit weights: what the binding lays out and refuses (CPU)."""
import os

import numpy as np
import pytest
import torch

from ragged_grouped_gemm_device_amd import moe as M

pytestmark = pytest.mark.skipif(not os.path.exists(M.LIB_PATH), reason="libmoe.so not built")


@pytest.mark.parametrize("form, per", [(M.MOE_X_BF16, 0), (M.MOE_X_MXFP8, 1), (M.MOE_X_MXFP4, 2)])
@pytest.mark.parametrize("act", [M.MOE_ACT_SWIGLU, M.MOE_ACT_SRELU])
def test_sized_shares_the_weights_alone(form, per, act):
    a = M.Experts4(8, 2, 16, 64, 96, act, form, device="cpu")
    b = a.sized(5)
    n1 = 192 if act == M.MOE_ACT_SWIGLU else 96
    assert a.w1_q.shape == (16, n1, 32) and a.w1_s.shape == (16, n1, 2) and a.w2_q.shape == (16, 64, 48) and a.w2_s.shape == (16, 64, 3)
    for name in ("w1_q", "w1_s", "w2_q", "w2_s"):
        assert getattr(a, name) is getattr(b, name)
    assert a.ws.data_ptr() != b.ws.data_ptr()
    for e, T in ((a, 8), (b, 5)):
        assert e.T == T
        if not per:
            assert e.x_q is None and e.a_s is None
            continue
        cap = M.moe_capacity_rows(T, 2, 16)
        assert e.x_q.shape == (T, 64 // per) and e.x_s.shape == (T, 2) and e.a_q.shape == (cap, 96 // per) and e.a_s.shape == (cap, 3)
    if per:
        assert a.a_q.data_ptr() != b.a_q.data_ptr() and a.x_q.data_ptr() != b.x_q.data_ptr()


def test_rows_that_a_routing_reaches():
    """No routing goes past them; some reach them."""
    rng = np.random.default_rng(0)
    for T, k, E in [(1, 1, 1), (1, 8, 256), (16, 8, 256), (5, 3, 4), (300, 2, 8), (129, 4, 4), (1021, 8, 32), (1 << 20, 8, 32)]:
        pairs, used = T * k, M._used_rows(T, k, E)
        assert used % M.MOE_ALIGN == 0 and used <= M.moe_capacity_rows(T, k, E)
        ends = []
        for trial in range(200 if T < 1 << 16 else 5):
            weight = np.full(E, 1 / E) if trial % 2 else rng.dirichlet(np.full(E, 0.1))
            counts = np.minimum(rng.multinomial(pairs, weight), T)
            ends.append(int((-(-counts // M.MOE_ALIGN) * M.MOE_ALIGN).sum()))
        assert max(ends) <= used
    assert M._used_rows(1, 8, 256) == 8 * M.MOE_ALIGN and M._used_rows(129, 4, 4) == 4 * 2 * M.MOE_ALIGN   # all of it


@pytest.mark.parametrize("kw, match", [
    (dict(mx=True), "mx"), (dict(fwd_stages=M.MOE_STAGE_FC1), "fwd_stages"), (dict(fwd_stages=0), "fwd_stages"), (dict(k=3), "k = 3"),
])
def test_forward_refuses_what_experts4_has_no_form_of(kw, match):
    kw = dict(kw)
    buf = M.Buffers(8, 2, 8, 64, 64, device="cpu")
    four = M.Experts4(8, kw.pop("k", 2), 8, 64, 64, device="cpu")
    for norms in (None, (M.BlockNorms(8, 64, device="cpu"), None, None, None)):
        with pytest.raises(ValueError, match=match):
            M.forward(buf, torch.zeros(8, 64), torch.zeros(8, 8), None, None, experts4=four, norms=norms, **kw)
    assert not buf.served


def test_sigmoid_routing_beside_the_softmax_balance_loss_is_refused():
    """The balance loss is that of softmax probabilities: beside sigmoid scores it would train the router towards
    another distribution than the one it routes by. The z loss takes any."""
    buf = M.Buffers(8, 2, 8, 64, 64, device="cpu")
    z = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t)  # noqa: E731
    for score, coef, refused in [(M.MOE_SCORE_SIGMOID, 1e-2, True), (M.MOE_SCORE_SIGMOID, 0.0, False), (M.MOE_SCORE_SOFTMAX, 1e-2, False)]:
        router = (M.Router(8, 64, 8, 2, balance_coef=coef, z_coef=1e-3, device="cpu"), z(64, 8))
        kw = dict(router=router, routing=M.Routing(score=score))
        match = "balance_coef" if refused else "GPU"   # off the GPU, where it is not refused before
        with pytest.raises(ValueError, match=match):
            M.forward(buf, z(8, 64), None, None, None, **kw)
        if refused:
            with pytest.raises(ValueError, match=match):
                M.backward(buf, z(8, 64), None, None, x_tokens=z(8, 64), **kw)


def test_a_gate_that_the_norms_were_not_made_for_has_no_silent_backward():
    z = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t)  # noqa: E731
    for cols, gate in ((0, z(8, 1)), (0, z(8, 64)), (1, z(8, 64)), (64, z(8, 1)), (1, None)):
        norms = M.BlockNorms(8, 64, cols, device="cpu")
        with pytest.raises(ValueError, match="gate"):
            norms.back_after(z(8, 64), z(64), gate, z(8, 64))
