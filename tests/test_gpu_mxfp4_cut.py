"""The products of 8-bit rows and 4-bit weights differ from exact ones by what the matrix cores cut off and by nothing
else: the products of 8 consecutive k are truncated at 2^-13 of the power of two that the largest sum of their operands'
exponents gives, and added up in fp32 (GPU). Bound against that sum: a group's place in the fp32 sum, 2^-23
of all magnitudes at most, for K / 8 groups and the joins of up to 16 partial sums, and half a step of bf16."""
import numpy as np
import pytest

from ._util import bf16_values
from .test_gpu_mxfp4 import M, Case  # noqa: F401

pytestmark = pytest.mark.gpu


def exponents(v):
    return np.where(v == 0, -200, np.frexp(v)[1] - 1)


def cut_products(x, w):
    """sum over groups of 8 of the truncated products of x [R, K] and w [N, K]."""
    p = (x[:, None] * w[None]).reshape(len(x), len(w), -1, 8)
    e = (exponents(x)[:, None] + exponents(w)[None]).reshape(p.shape).max(3, keepdims=True)
    step = np.ldexp(1.0, e - 13)
    return (np.trunc(p / step) * step).sum((2, 3))


def test_a_product_below_the_groups_last_place_is_cut():
    """On the host: 256 + 2^-5 stays, 256 + 1.75 * 2^-6 is 256 (x = 16 and 2^-3, w = 16 and 2^-2 ...)."""
    one = np.zeros((1, 8))
    x, w = one.copy(), one.copy()
    x[0, :2], w[0, :2] = (16.0, 0.125), (16.0, 0.25)
    assert cut_products(x, w)[0, 0] == 256 + 2.0**-5
    x[0, 1] = 1.75 * 2.0**-4
    assert cut_products(x, w)[0, 0] == 256
    w[0, 0], x[0, 0] = 1.5, 1.5   # 2.25: the exponents' sum is 0, not 1
    x[0, 1], w[0, 1] = 2.0**-7, 2.0**-6
    assert cut_products(x, w)[0, 0] == 2.25 + 2.0**-13


@pytest.mark.parametrize("counts, K, N, gather", [
    ([3, 0, 16, 9], 544, 72, False), ([17, 1, 0, 24], 2080, 136, True), ([40, 64, 0, 33, 1], 512, 264, True),
    ([129, 0, 70, 200], 192, 264, False), ([300, 257, 0, 31], 160, 520, True),
])
def test_the_difference_is_the_cut_off(M, counts, K, N, gather):  # noqa: F811
    c = Case(M, counts, K, N, M.MOE_X_MXFP8, gather)
    got = bf16_values(c.run("none"))
    for e, n in enumerate(counts):
        w = c.wv[e]
        for r in range(c.offsets[e], c.offsets[e] + n, 32):
            x = c.rows[r:min(r + 32, c.offsets[e] + n)]
            y, ref = got[r:r + len(x)], cut_products(x, w)
            sums = (K // 8 + 16) * 2.0**-23 * (np.abs(x) @ np.abs(w).T)
            assert (np.abs(y - ref) <= sums + 2.0**-8 * (np.abs(ref) + sums)).all(), (e, r)
