"""Experts served on 4-bit weights: the chain of both products, each from the codes that the run itself made of its
rows, and several token counts and streams on one set of weights (GPU).

Bounds of a product: sums of K terms in fp32, K * 2^-22 of their magnitudes; with 8-bit rows 7 * 2^-13 of the largest product of
each 8 as well (the matrix cores cut smaller ones off there); the activation's, with |f'| <= 1.13; half a step of bf16."""
import numpy as np
import pytest
import torch

from oracle import block_oracle as B
from oracle import dense_oracle as D
from oracle import moe_oracle as O

from ._util import bf16_values

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def M():
    from ragged_grouped_gemm_device_amd import moe
    moe.load()
    return moe


class Served:
    """Tokens, their routing and the experts' buffers for one Experts4."""

    def __init__(self, M, four, seed=0):
        T, k = four.T, four.k
        E, d, n = four.w2_q.shape[0], four.w2_q.shape[1], 2 * four.w2_q.shape[2]
        self.M, self.four = M, four
        self.buf = M.Buffers(T, k, E, d, n, gated=four.act in M._GATED)
        g = torch.Generator("cuda").manual_seed(seed + T)
        self.x = torch.randn(T, d, device="cuda", generator=g).to(BF)
        self.logits = torch.randn(T, E, device="cuda", generator=g)
        self.routing = M.Routing()

    def run(self):
        self.M.forward(self.buf, self.x, self.logits, None, None, routing=self.routing, experts4=self.four)
        return self.buf.out


def weights(M, T, k, E, d, n, act, form):
    four = M.Experts4(T, k, E, d, n, D.ACTS.index(act), form)
    g = torch.Generator("cuda").manual_seed(d + n)
    n1 = 2 * n if act in D.GATED else n
    four.load((torch.randn(E, d, n1, device="cuda", generator=g) * d**-0.5).to(BF),
              (torch.randn(E, n, d, device="cuda", generator=g) * n**-0.5).to(BF))
    return four


def product(x, w, act, form):
    """f(x w^T) in 64 bits and how far off it may come out."""
    z = x @ w.T
    dz = x.shape[1] * 2.0**-22 * (np.abs(x) @ np.abs(w).T)
    if form == 1:
        eights = lambda v: np.abs(v).reshape(v.shape[0], -1, 8).max(2)  # noqa: E731
        dz = dz + 7 * 2.0**-13 * (eights(x) @ eights(w).T)
    ref = D.act_forward(z, act)
    if act in D.GATED:   # |f'| <= 1.13 for both gates, |f(g)| <= |g|
        (g, u), (dg, du) = O.deinterleave(z), O.deinterleave(dz)
        slack = 1.13 * dg * np.abs(u) + (np.abs(g) + 1.13 * dg) * du + 8 * 2.0**-23 * np.abs(g * u)
    elif act == "srelu":
        slack = 2 * np.abs(z) * dz + dz * dz
    else:
        slack = 1.13 * dz + 8 * 2.0**-23 * np.abs(z)
    return ref, slack + 2.0**-8 * (np.abs(ref) + slack)


@pytest.mark.parametrize("form", [0, 1, 2])
@pytest.mark.parametrize("T, k, E, d, n, act", [
    (1, 2, 8, 128, 64, "swiglu"), (37, 4, 16, 192, 128, "geglu"), (300, 2, 8, 320, 192, "swiglu"), (600, 3, 4, 256, 64, "srelu"),
])
def test_the_chain_from_the_runs_own_codes(M, form, T, k, E, d, n, act):
    s = Served(M, weights(M, T, k, E, d, n, act, form))
    s.run()
    torch.cuda.synchronize()
    b, four = s.buf, s.four
    c = lambda t: t.cpu().numpy()  # noqa: E731
    counts, offsets = c(b.counts), c(b.offsets)
    live = np.concatenate([np.arange(o, o + m) for o, m in zip(offsets, counts)])
    of_token = c(b.src_of)[live] // k

    def rows(v, q, sc, at):
        """The values that the product read, from the codes; those are the oracle's of the bf16 rows v."""
        if form == 0:
            return v
        q, sc = c(q)[at], c(sc)[at]
        if form == 1:
            want = O.quant_mxfp8(v, colwise=False)
        else:
            want = B.quant_mxfp4(v)
            want = B.pack4(want[0]), want[1]
        assert np.array_equal(q, want[0]) and np.array_equal(sc, want[1])
        return O.mx_dequant(q, sc) if form == 1 else B.dequant_mxfp4(q, sc)

    x = rows(bf16_values(s.x), four.x_q, four.x_s, slice(None))[of_token]
    a = rows(bf16_values(b.a)[live], four.a_q, four.a_s, live)
    w1, w2 = (B.dequant_mxfp4(c(q), c(sc)) for q, sc in ((four.w1_q, four.w1_s), (four.w2_q, four.w2_s)))
    expert = np.repeat(np.arange(E), counts)
    for v, w, f, got in ((x, w1, act, b.a), (a, w2, "none", b.y)):
        got = bf16_values(got)[live]
        for e in np.flatnonzero(counts):
            at = expert == e
            ref, off = product(v[at], w[e], f, form)
            assert (np.abs(got[at] - ref) <= off).all(), (f, e)
    # sums of k terms in fp32, rounded to bf16
    y = np.zeros((b.M_cap, d))
    y[live] = bf16_values(b.y)[live]
    w = c(b.topk_w).astype(np.float64)
    ref, most = (O.combine(v, c(b.row_of), k, w, rounding=False) for v in (y, np.abs(y)))
    assert (np.abs(bf16_values(b.out) - ref) <= 2.0**-8 * np.abs(ref) + 2 * k * 2.0**-24 * most).all()


@pytest.mark.parametrize("form", [0, 1, 2])
def test_token_counts_and_streams_on_one_set_of_weights(M, form):
    """A prompt and decode steps on the same weights, alone, at once on two streams, and one of them from a graph."""
    prompt = weights(M, 150, 2, 8, 192, 128, "swiglu", form)
    step, other = prompt.sized(3), prompt.sized(150)
    assert step.w1_q is prompt.w1_q and step.w2_s is prompt.w2_s and (step.T, prompt.T) == (3, 150)
    calls = [Served(M, f, i) for i, f in enumerate((prompt, step, other))]
    want = [s.run().clone() for s in calls]
    apart = weights(M, 3, 2, 8, 192, 128, "swiglu", form)
    single = Served(M, apart, 1)
    assert torch.equal(single.run(), want[1])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        calls[1].run()
    streams = [torch.cuda.Stream() for _ in calls]
    for rep in range(4):
        for s in calls:
            s.buf.out.zero_()
        torch.cuda.synchronize()
        for i, (st, s) in enumerate(zip(streams, calls)):
            with torch.cuda.stream(st):
                g.replay() if i == 1 else s.run()
        torch.cuda.synchronize()
        for s, w in zip(calls, want):
            assert torch.equal(s.buf.out, w), rep
    # weights loaded into one are there for all
    step.load(torch.ones(8, 192, 256, dtype=BF, device="cuda"), torch.ones(8, 128, 192, dtype=BF, device="cuda"))
    assert not torch.equal(calls[0].run(), want[0])


def test_another_token_count_is_refused(M):
    s = Served(M, weights(M, 8, 2, 8, 64, 64, "swiglu", 0))
    s.x = s.x[:4].contiguous()
    s.logits = s.logits[:4].contiguous()
    with pytest.raises(ValueError, match="expected"):
        s.run()


@pytest.mark.parametrize("form", [1, 2])
def test_codes_past_the_rows_that_a_routing_reaches_are_left(M, form):
    """One token and 64 experts: its 4 rows lie in the first 4 regions, not in the capacity for any routing."""
    s = Served(M, weights(M, 1, 4, 64, 64, 64, "swiglu", form))
    want = s.run().clone()
    used = int(s.buf.offsets[-1])
    assert used == 4 * M.MOE_ALIGN < s.buf.M_cap / 16
    for t in (s.four.a_q, s.four.a_s):
        t.fill_(0x55)
    assert torch.equal(s.run(), want)
    for t in (s.four.a_q, s.four.a_s):
        assert (t[used:] == 0x55).all()
