"""Experts served on 4-bit weights: several token counts and streams on one set of weights (GPU)."""
import pytest
import torch

from oracle import dense_oracle as D

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
