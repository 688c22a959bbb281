"""4-bit blocks and the experts' products with them, against the oracle (GPU).

Products: fp32 sums of K terms that a matrix instruction may truncate, K 2^-22 of the sum of their
magnitudes, and a bf16 rounding, 2^-8 of the result. The instruction for 8- and 4-bit operands first adds groups of 8
consecutive products as whole numbers of 2^-13 of the power of two under the largest, cut off (256 + 2^-5 is kept, 256 +
1.75 * 2^-6 is 256). Two 4-bit values' products are multiples of 1/4 and at most 36 = 2.25 * 2^2 * 2^2, whose unit is 2^-9: nothing
is lost. With 8-bit rows the 7 others lose less than a unit each: 7 * 2^-13 of the largest, which is at most the
largest |x| times the largest |w| of the 8."""
import numpy as np
import pytest
import torch

from oracle import block_oracle as B
from oracle import dense_oracle as D
from oracle import moe_oracle as O

from ._util import bf16_tensor, bf16_values

pytestmark = pytest.mark.gpu
BF, U8, I32 = torch.bfloat16, torch.uint8, torch.int32


@pytest.fixture(scope="module")
def M():
    from ragged_grouped_gemm_device_amd import moe
    moe.load()
    return moe


def u8(*shape):
    return torch.full(shape, 99, dtype=U8, device="cuda")


def quant(M, x):
    """Row-wise codes and scales of x [.., R, C]."""
    q, s = u8(*x.shape[:-1], x.shape[-1] // 2), u8(*x.shape[:-1], x.shape[-1] // 32)
    M.moe_quant_mxfp4(x, M.MOE_QUANT_ROWWISE, q, s)
    return q, s


def test_every_bf16_value_under_every_scale_that_holds_it(M):
    """All 65536 patterns, each block led by its own largest magnitude and by ones up to 2^9 larger: codes and scales
    bit for bit; blocks with a NaN or an infinity are NaN whole."""
    bits = np.arange(65536, dtype=np.uint32)
    for up in (0, 1, 2, 4, 9):
        lead = np.minimum((bits & 0x7fff) + 128 * up, np.where((bits & 0x7fff) < 0x7f80, 0x7f7f, 0x7fff))
        v = np.zeros((65536, 32), np.uint16)
        v[:, 3], v[:, 17] = bits, lead
        x = bf16_tensor(v)
        q, s = quant(M, x)
        val = bf16_values(x)
        some = np.r_[0:65536:97, 0x7f70:0x7fa0, 0xff70:0xffa0, 0:40]      # the oracle walks block by block
        rq, rs = B.quant_mxfp4(val[some])
        assert np.array_equal(s.cpu().numpy()[some], rs)
        assert np.array_equal(q.cpu().numpy()[some], B.pack4(rq))
        out = torch.empty(65536, 32, dtype=BF, device="cuda")
        M.moe_dequant_mxfp4(q, s, out)
        want = B.dequant_mxfp4(q.cpu().numpy(), s.cpu().numpy())
        # a largest value above 1.75 * 2^127 takes scale 2^126 and code 4: 2^128, past bf16's numbers
        want = np.where(np.abs(want) >= 2.0**128, np.copysign(np.inf, want), want)
        got = bf16_values(out)
        assert np.array_equal(np.isnan(got), np.isnan(want))
        fine = ~np.isnan(want)
        off = np.flatnonzero(got[fine] != want[fine])
        assert not len(off), (len(off), got[fine][off[:4]], want[fine][off[:4]])   # code times scale is a bf16 number, subnormals too
        # every finite block: off by half a step at most
        fin = np.isfinite(val).all(1) & ~np.isinf(want).any(1)
        step = np.exp2(s.cpu().numpy()[fin, 0].astype(float) - 127)[:, None]
        err, mag = np.abs(want[fin] - val[fin]), np.abs(val[fin])
        assert (err <= np.maximum(mag / 4, step / 4)).all()


@pytest.mark.parametrize("batch, R, C", [(1, 32, 8), (1, 64, 72), (3, 96, 200), (2, 256, 64), (1, 512, 320), (1, 2880, 96), (2, 288, 1032)])
def test_transposed_is_the_row_wise_of_the_transposed(M, batch, R, C):
    x = (torch.randn(batch, R, C, device="cuda") * torch.exp(2 * torch.randn(batch, 1, C, device="cuda"))).to(BF)
    x[0, 5, 3] = float("inf")
    q, s = u8(batch, C, R // 2), u8(batch, C, R // 32)
    M.moe_quant_mxfp4(x, M.MOE_QUANT_COLWISE, q_col=q, s_col=s)
    rq, rs = quant(M, x.transpose(1, 2).contiguous())
    assert torch.equal(q, rq) and torch.equal(s, rs)
    if C % 32 == 0:
        both = [u8(batch, R, C // 2), u8(batch, R, C // 32), u8(batch, C, R // 2), u8(batch, C, R // 32)]
        M.moe_quant_mxfp4(x, M.MOE_QUANT_ROWWISE | M.MOE_QUANT_COLWISE, *both)
        assert torch.equal(both[2], q) and torch.equal(both[3], s)
        assert all(torch.equal(a, b) for a, b in zip(both, quant(M, x)))


def test_scales_at_any_byte(M):
    """Scale arrays that start at odd addresses."""
    x = torch.randn(256, 64, device="cuda").to(BF)
    q, s = u8(64, 128), u8(64 * 8 + 1)[1:].view(64, 8)
    M.moe_quant_mxfp4(x, M.MOE_QUANT_COLWISE, q_col=q, s_col=s)
    rq, rs = quant(M, x.t().contiguous())
    assert torch.equal(q, rq) and torch.equal(s, rs)


# ---------------------------------------------------------------- products
class Case:
    """Experts with given row counts: x (padding rows NaN), weights, and the oracle's values of both."""

    def __init__(self, M, counts, K, N, form, gather, k=2, seed=0, T=None):
        self.M, self.counts, self.K, self.N, self.form = M, counts, K, N, form
        E = len(counts)
        pairs = sum(counts)
        self.T = T or max(max(counts), -(-pairs // k))
        assert max(counts) <= self.T and pairs <= self.T * k
        self.k, self.E = k, E
        g = torch.Generator("cuda").manual_seed(seed + K + N)
        cap = M.moe_capacity_rows(self.T, k, E)
        self.offsets = np.concatenate([[0], np.cumsum([-(-c // 128) * 128 for c in counts])]).astype(np.int32)
        live = np.concatenate([np.arange(o, o + c) for o, c in zip(self.offsets, counts)]).astype(np.int64)
        rng = np.random.default_rng(seed)
        tokens = rng.integers(0, self.T, len(live))
        self.src_of = np.full(cap, -1, np.int32)
        self.src_of[live] = tokens * k
        x = torch.randn(self.T if gather else cap, K, device="cuda", generator=g).to(BF)
        if not gather:
            pad = np.setdiff1d(np.arange(cap), live)
            x[torch.from_numpy(pad).cuda()] = float("nan")
        self.xs = None
        if form == M.MOE_X_MXFP4:
            self.x, self.xs = quant(M, x)
            xv = B.dequant_mxfp4(self.x.cpu().numpy(), self.xs.cpu().numpy())
        elif form == M.MOE_X_MXFP8:
            self.x, self.xs = u8(*x.shape), u8(x.shape[0], K // 32)
            M.moe_quant_mxfp8(x.nan_to_num(), M.MOE_QUANT_ROWWISE, self.x, self.xs)
            if not gather:
                self.x[torch.from_numpy(pad).cuda()] = 0x7f   # E4M3's NaN
            xv = O.mx_dequant(self.x.cpu().numpy(), self.xs.cpu().numpy())
        else:
            self.x = x
            xv = bf16_values(x)
        w = (torch.randn(E, N, K, device="cuda", generator=g) * K**-0.5).to(BF)
        self.w_q, self.w_s = quant(M, w)
        self.wv = B.dequant_mxfp4(self.w_q.cpu().numpy(), self.w_s.cpu().numpy())
        self.rows = np.zeros((cap, K))
        self.rows[live] = xv[tokens] if gather else xv[live]
        self.live, self.cap, self.gather = live, cap, gather
        self.ws = u8(max(16, M.moe_grouped_linear_mxfp4_workspace_bytes(self.T, k, E, K, N)))
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        self.d_off, self.d_cnt, self.d_src = dev(self.offsets), dev(np.asarray(counts, np.int32)), dev(self.src_of)

    def new_y(self, act):
        y = torch.empty(self.cap, self.N // 2 if act in D.GATED else self.N, dtype=BF, device="cuda")
        return y.fill_(-123.0)

    def run(self, act, y=None, ws=None):
        y = self.new_y(act) if y is None else y
        self.M.moe_grouped_linear_mxfp4(self.x, self.w_q, self.w_s, self.d_off, self.d_cnt, y, self.T, self.k, act=D.ACTS.index(act),
                                        x_s=self.xs, src_of=self.d_src if self.gather else None, workspace=self.ws if ws is None else ws)
        return y

    def cut_off(self, a, w):
        """What 8-bit rows' products lose."""
        eights = lambda v: np.abs(v).reshape(v.shape[0], -1, 8).max(2)  # noqa: E731
        return 7 * 2.0**-13 * (eights(a) @ eights(w).T) if self.form == self.M.MOE_X_MXFP8 else 0

    def check(self, act):
        y = self.run(act)
        got = bf16_values(y)
        dead = np.setdiff1d(np.arange(self.cap), self.live)
        assert (got[dead] == -123.0).all(), "a row past its expert's was written"
        for e, c in enumerate(self.counts):
            if not c:
                continue
            a = self.rows[self.offsets[e]:self.offsets[e] + c]
            z = a @ self.wv[e].T
            dz = self.K * 2.0**-22 * (np.abs(a) @ np.abs(self.wv[e]).T) + self.cut_off(a, self.wv[e])     # error of z
            ref = D.act_forward(z, act)
            if act in D.GATED:   # |f'| <= 1.13 for both gates, |f(g)| <= |g|
                g, u = O.deinterleave(z)
                dg, du = O.deinterleave(dz)
                slack = 1.13 * dg * np.abs(u) + (np.abs(g) + 1.13 * dg) * du + 8 * 2.0**-23 * np.abs(g * u)
            elif act == "srelu":
                slack = 2 * np.abs(z) * dz + dz * dz
            else:
                slack = 1.13 * dz + 8 * 2.0**-23 * np.abs(z)
            off = np.abs(got[self.offsets[e]:self.offsets[e] + c] - ref)
            assert (off <= slack + 2.0**-8 * (np.abs(ref) + slack)).all(), (act, e, c, float(off.max()))


FORMS = ["bf16", "mxfp8", "mxfp4"]
# mean rows an expert from one to hundreds, each with empty experts, and ends inside a tile
COUNTS = {
    "one": [0, 1, 0, 1, 1], "few": [3, 0, 16, 17, 9], "dozens": [40, 1, 0, 33, 64], "tens": [70, 65, 0, 128, 1, 60],
    "hundred": [129, 0, 127, 200, 1, 300], "hundreds": [256, 511, 0, 1, 257, 700],
}


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("rows", list(COUNTS))
@pytest.mark.parametrize("K, N, act, gather", [
    (32, 8, "none", False), (96, 64, "swiglu", True), (160, 264, "silu", True), (512, 320, "geglu", False), (544, 72, "gelu", True),
    (1056, 128, "srelu", False), (2880, 192, "swiglu", True),
])
def test_products(M, form, rows, K, N, act, gather):
    Case(M, COUNTS[rows], K, N, FORMS.index(form), gather, seed=len(rows)).check(act)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("mean", [40, 100, 300])
@pytest.mark.parametrize("K, N, act, gather", [
    (32, 1288, "none", False), (96, 1344, "swiglu", True), (544, 1544, "gelu", True), (1056, 1408, "geglu", False), (2208, 1800, "srelu", True),
])
def test_products_of_many_tiles(M, form, mean, K, N, act, gather):
    """As many tokens and columns as make tiles of 64, 128 and 256 rows worth while, whatever the counts are then."""
    counts = [3, 0, 16, 17, 9, 70, 65, 0, 128, 1, 60, 300] + [0] * 8 + [2, 0]
    Case(M, counts, K, N, FORMS.index(form), gather, T=len(counts) * mean // 2).check(act)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("counts, K, N, act", [
    ([3, 0, 1, 7], 9248, 136, "none"),               # few columns: K in eighths, and past the scales that LDS holds
    ([2, 0, 5, 1] * 5 + [9], 9248, 1088, "swiglu"),  # many: in quarters
    ([17, 0, 33, 9, 20], 9248, 320, "gelu"),         # 32 rows at a time
])
def test_few_rows_of_a_long_width(M, form, counts, K, N, act):
    Case(M, counts, K, N, FORMS.index(form), True).check(act)


@pytest.mark.parametrize("form", FORMS)
def test_many_tiles_a_workgroup(M, form):
    """More tiles than compute units, so that workgroups walk on; widths that end inside a tile."""
    c = Case(M, [300, 257, 1, 0, 1000, 640, 30], 192, 13 * 256 + 8, FORMS.index(form), True)
    c.check("none")
    c = Case(M, [3, 1, 0, 2] * 30, 288, 1600, FORMS.index(form), False)
    c.check("swiglu")


def test_more_experts_than_lanes(M):
    """130 experts with a row here and there."""
    counts = [0] * 130
    for e in (0, 63, 64, 65, 100, 129):
        counts[e] = 1 + e % 3
    for form in range(3):
        Case(M, counts, 256, 64, form, True).check("none")


def test_blocks_that_are_nan(M):
    """A weight block's NaN scale makes its column NaN in that expert alone; so does a row's."""
    for counts in (COUNTS["few"], COUNTS["hundreds"]):
        for form in range(3):
            c = Case(M, counts, 160, 64, form, False)
            c.w_s[2, 7, 3] = 255
            if c.xs is not None:
                c.xs[int(c.offsets[3]), 1] = 255
            y = bf16_values(c.run("none"))
            bad = np.zeros(y.shape, bool)
            bad[c.offsets[2]:c.offsets[2] + counts[2], 7] = True
            if c.xs is not None and counts[3]:
                bad[c.offsets[3]] = True
            assert np.array_equal(np.isnan(y[c.live]), bad[c.live])


def test_largest_and_smallest_scales(M):
    """Scales whose product leaves fp32's normal range in either operand come out as the exact values do."""
    for counts in (COUNTS["few"], COUNTS["hundred"]):
        for form in range(3):
            c = Case(M, counts, 64, 64, form, False)
            w_s = c.w_s.clone()
            for up in (-100, 100):
                c.w_s.copy_((w_s.int() + up).to(U8))
                got = bf16_values(c.run("none"))[c.live]
                c.w_s.copy_(w_s)
                base = bf16_values(c.run("none"))[c.live]
                assert np.array_equal(got, base * 2.0**up)


@pytest.mark.parametrize("rows", ["few", "tens", "hundreds"])
def test_captured_and_on_two_streams(M, rows):
    a, b = (Case(M, COUNTS[rows], 544, 320, f, True) for f in (0, 2))
    ya, yb = a.run("geglu"), b.run("none")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.run("geglu", ya)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for rep in range(3):
        a.x.copy_(torch.randn(a.x.shape, device="cuda"))
        want_a, want_b = a.run("geglu", ws=a.ws.clone()), b.run("none")
        ya.fill_(-123.0)
        yb.fill_(-123.0)
        torch.cuda.synchronize()
        with torch.cuda.stream(streams[0]):
            g.replay()
        with torch.cuda.stream(streams[1]):
            b.run("none", yb)
        torch.cuda.synchronize()
        assert torch.equal(ya, want_a) and torch.equal(yb, want_b), rep


def test_a_long_expert_buffer(M):
    """Rows of the experts' buffer past 2^31 bytes (the last expert's)."""
    E, k, K, N = 2, 1, 8192, 64
    T = 140000
    cap = M.moe_capacity_rows(T, k, E)
    counts = [139776, 200]
    off = torch.tensor([0, 139776, 140032], dtype=I32, device="cuda")
    x = torch.zeros(cap, K, dtype=BF, device="cuda")
    tail = torch.randn(200, K, device="cuda").to(BF)
    x[139776:139976] = tail
    w = (torch.randn(E, N, K, device="cuda") * K**-0.5).to(BF)
    w_q, w_s = quant(M, w)
    y = torch.empty(cap, N, dtype=BF, device="cuda")
    ws = u8(max(16, M.moe_grouped_linear_mxfp4_workspace_bytes(T, k, E, K, N)))
    M.moe_grouped_linear_mxfp4(x, w_q, w_s, off, torch.tensor(counts, dtype=I32, device="cuda"), y, T, k, workspace=ws)
    a, b = bf16_values(tail), B.dequant_mxfp4(w_q[1].cpu().numpy(), w_s[1].cpu().numpy())
    ref = a @ b.T
    assert (np.abs(bf16_values(y[139776:139976]) - ref) <= 2.0**-8 * np.abs(ref) + K * 2.0**-22 * (np.abs(a) @ np.abs(b).T)).all()
    assert (y[:139776] == 0).all()
