"""Which form of the dense products the tests' shapes take, by the library's own plan (CPU): every form
that the plan chooses for some shape is run by a GPU test, and no launch has 2^32 threads."""
import os
import random
import shutil
import subprocess

import pytest

from . import test_gpu_dense, test_gpu_dense_forms, test_gpu_dense_shapes

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "ragged_grouped_gemm_device_amd", "csrc")
CXX = shutil.which("g++") or shutil.which("c++")
pytestmark = pytest.mark.skipif(CXX is None, reason="no host compiler")
FORWARD, DGRAD, WGRAD = range(3)
MAIN = r"""
#include <cstdio>
#include "dense_plan.hpp"
int main() {
    long long M, N, K, out;
    int pass;
    while (scanf("%lld %lld %lld %d %lld", &M, &N, &K, &pass, &out) == 5) {
        const moe::DensePlan d = moe::dense_plan(M, N, K, (moe::DensePass)pass);
        printf("%c %d %d %d %d %d %d\n", d.kind, d.ntm, d.ntn, d.splits, d.tail_first, d.tail_splits,
               d.splits > 1 && moe::dense_join_wide(M * (out / 8), d.splits));
    }
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    at = tmp_path_factory.mktemp("plan")
    (at / "plan.cpp").write_text(MAIN)
    subprocess.run([CXX, "-O1", "-std=c++17", "-I", CSRC, str(at / "plan.cpp"), "-o", str(at / "plan")], check=True)

    def run(products):
        r = subprocess.run([str(at / "plan")], input="\n".join("%d %d %d %d %d" % p for p in products), text=True,
                           capture_output=True, check=True)
        return [(line[0], *map(int, line.split()[1:])) for line in r.stdout.splitlines()]
    return run


def _products(shapes, gated=False):
    """(rows, columns, reduction, pass, output columns) of the products of T x K x N layers."""
    if gated:
        return [(T, N, K, FORWARD, N // 2) for T, K, N in shapes]
    return [p for T, K, N in shapes for p in ((T, N, K, FORWARD, N), (T, K, N, DGRAD, K), (K, N, T, WGRAD, N))]


def _forms(plan, products):
    """Kernel, pieces of K and join of each product, as dense.hip launches them."""
    out = []
    for (M, _, _, which, _), (kind, _, _, splits, _, tail, wide) in zip(products, plan(products)):
        rows = next(r for r in (8, 16, 32, 64) if M <= r or r == 64) if kind == "s" and which != WGRAD else 0
        out.append((which, kind, rows, "last round" if tail > 1 else "split" if splits > 1 else "whole", wide))
    return out


def _sample(step, n=20000):
    rng = random.Random(11)
    log = lambda lo, hi, step=1: max(step, int(lo * (hi / lo) ** rng.random()) // step * step)  # noqa: E731
    return [(log(1, 32768), log(8, 8192, 8), log(step, 8192, step)) for _ in range(n)]


def _missing(plan, products, tested, reduce=lambda form: form):
    ours = {reduce(f) for f in _forms(plan, tested)}
    out = {}
    for p, form in zip(products, _forms(plan, products)):
        if reduce(form) not in ours:
            out.setdefault(reduce(form), p[:3])
    return out


def test_every_form_that_the_plan_chooses_is_run_by_a_gpu_test(plan):
    some = range(48 + len(test_gpu_dense_shapes.CHOSEN))
    shapes = ([test_gpu_dense_shapes._shape(random.Random(i), i) for i in some] + test_gpu_dense.SHAPES
              + test_gpu_dense_forms.FORMS)
    assert not _missing(plan, _products(_sample(8)), _products(shapes))


@pytest.mark.parametrize("gated", [False, True])
def test_every_form_of_the_forward_is_run_with_every_activation(plan, gated):
    """A split product leaves its activation to the joining kernel, whatever its tiles are."""
    reduce = lambda f: ("split", f[4]) if f[3] == "split" else f  # noqa: E731
    shapes = test_gpu_dense.SHAPES + test_gpu_dense_forms.FORWARD
    sample = _products(_sample(64 if gated else 8), gated)
    assert not _missing(plan, [p for p in sample if p[3] == FORWARD], [p for p in _products(shapes, gated) if p[3] == FORWARD],
                        reduce)


def test_the_shapes_take_the_forms_they_stand_for(plan):
    form = lambda T, K, N, which: _forms(plan, _products([(T, K, N)]))[which][1:]  # noqa: E731
    assert form(10959, 3360, 320, FORWARD) == ("H", 0, "whole", 0)
    assert form(5597, 1648, 272, WGRAD) == ("M", 0, "split", 0)
    assert form(1812, 192, 6280, WGRAD) == ("D", 0, "split", 0)
    assert form(25424, 3064, 784, WGRAD) == ("L", 0, "split", 0)
    assert form(8192, 2880, 5760, WGRAD) == ("L", 0, "last round", 0)
    assert form(1, 8192, 4096, FORWARD) == ("s", 8, "split", 1)


def test_no_launch_reaches_2_to_the_32_threads(plan):
    """Past that a launch is cut off without an error. Operands and partial sums within 288 GB."""
    rng = random.Random(12)
    log = lambda lo, hi, step: max(step, int(lo * (hi / lo) ** rng.random()) // step * step)  # noqa: E731
    products = []
    while len(products) < 20000:
        T, K, N = log(1 << 12, 1 << 30, 1), log(8, 1 << 20, 8), log(8, 1 << 20, 8)
        if 2 * (T * K + K * N + T * N) <= 288 << 30 and (T + 127) // 128 * ((max(K, N) + 127) // 128) < 1 << 30:
            products += _products([(T, K, N)])
    threads = {"s": 256, "M": 256, "D": 256, "H": 512, "L": 512}
    at_once = {"M": 512, "L": 256}   # persistent: no more workgroups than these
    for p, (kind, ntm, ntn, splits, _, _, wide) in zip(products, plan(products)):
        blocks = ntm * ntn * splits
        assert min(blocks, at_once.get(kind, blocks)) * threads[kind] < 1 << 32, p
        if splits > 1:
            assert p[0] * p[4] // 8 * (8 if wide else 1) + 256 < 1 << 32, p
            assert 4 * splits * p[0] * p[1] <= 288 << 30, p
