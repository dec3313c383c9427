"""orthogonalize's error against the iteration in 64 bits, as sharp as its arithmetic.

The result's rounding to bf16 is at most 2^-8 of an element and 1.66e-3 in the relative
Frobenius norm of many, held to 2^-9.  Sides up to 64 carry every operand as a pair of
fp16, 22 bits: 2^-22 of the norm, magnified a^5 = 485 times at most in the weakest
directions, is d = 1.2e-4, and nothing next to the rounding of many elements.  Of few
elements the error is that of rounding the exact result, and at most 2 d more (an element
beside a tie goes to the other neighbour).
Longer sides round X and the square matrices' elements off the diagonal to fp16 (what
that leaves of a diagonal is put back).  The same iteration in 64 bits with those
roundings and no others, run on the CPU before any of this on a GPU, is off by 1.75e-3
(long matrices) to 2.04e-3 (square ones of 66 to 256, 20 seeds): held to 2.2e-3.  With
other coefficients, whose maps have steeper slopes, the bound is that simulation's error
for the matrix and a quarter more; without a diagonal put back it is 1.4 to 3 times it.
"""
import pytest
import torch

import mx_block_quantization_gb300 as mxq
from tests.gpu_util import require_gpu
from tests.test_gpu_orthogonalize import COEFFICIENTS, iteration, momentum, off

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    yield
    assert mxq.device_status(clear=True) == 0


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("batch,m,n,pad", [
    (1, 64, 64, 0), (3, 48, 48, 0), (2, 50, 33, 3), (1, 17, 1000, 0), (1, 64, 8192, 0), (2, 40, 9000, 0), (1, 9000, 40, 0),
    (1, 8192, 64, 0), (4, 8, 8, 0), (1, 63, 64, 0), (2, 64, 300, 8), (1, 400, 56, 1), (5, 16, 16, 0),
])
def test_sides_up_to_64_are_exact_to_the_rounding(batch, m, n, pad, kind):
    for seed in range(4):
        g = momentum(batch, m, n, kind, pad, seed)
        assert off(mxq.orthogonalize(g), iteration(g)) <= 2.0**-9


@pytest.mark.parametrize("m,n", [(1, 1), (1, 7), (9, 1), (2, 3), (31, 5), (1, 3000), (513, 2), (3, 20000)])
def test_smallest_sides_are_exact_to_the_rounding(m, n):
    for seed in range(4):
        g = momentum(1, m, n, seed=seed)[0] + 1e-4
        want = iteration(g)
        assert off(mxq.orthogonalize(g), want) <= off(want.float().bfloat16(), want) + 2.4e-4


@pytest.mark.parametrize("co", [(1.5, -0.5, 0.0), (1.6, -0.65, 0.05)])
@pytest.mark.parametrize("m,n", [(64, 40), (20, 30), (64, 8192)])
def test_pairs_with_an_addend(m, n, co):
    g = momentum(1, m, n)
    assert off(mxq.orthogonalize(g, coefficients=co), iteration(g, coefficients=co)) <= 2.0**-9


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("batch,m,n,pad", [
    (1, 65, 70, 0), (1, 66, 66, 0), (1, 100, 100, 0), (1, 128, 256, 0), (1, 256, 128, 0), (1, 256, 256, 0), (2, 200, 333, 0),
    (1, 333, 200, 3), (1, 257, 511, 5), (1, 520, 264, 8), (1, 700, 1300, 0), (1, 1301, 703, 0), (40, 96, 160, 0),
    (2, 512, 2048, 0), (1, 2000, 640, 0), (1, 65, 8192, 3), (1, 300, 5000, 0), (1, 5001, 300, 0), (3, 128, 6000, 8),
    (1, 520, 12000, 0),
])
def test_longer_sides(batch, m, n, pad, kind):
    g = momentum(batch, m, n, kind, pad)
    assert off(mxq.orthogonalize(g), iteration(g)) <= 2.2e-3


def with_rounded_operands(g, steps, coefficients, eps=1e-7):
    a, b, c = coefficients

    def half(x):
        f, e = torch.frexp(x)
        return torch.ldexp(torch.round(f * 2048) / 2048, e)

    def beside_the_diagonal(x):
        d = torch.diag(x.diagonal())
        return half(x - d) + d

    x = g.double().cpu()
    wide = x.shape[0] <= x.shape[1]
    x = half((x if wide else x.T) / (x.norm() + eps))
    one = torch.eye(x.shape[0], dtype=torch.float64)
    for s in range(steps):
        q = beside_the_diagonal(x @ x.T)
        x = beside_the_diagonal(a * one + b * q + c * q @ q) @ x
        x = half(x) if s + 1 < steps else x.float().bfloat16().double()
    return x if wide else x.T


@pytest.mark.parametrize("co,steps,m,n", [
    ((2.9, -3.0, 0.7), 5, 70, 8000), ((2.5, -1.9, 0.0), 5, 4160, 256), ((2.5, -1.9, 0.0), 8, 70, 8000),
    ((2.5, -1.9, 0.0), 8, 4160, 256), ((2.6, -2.5, 0.4), 8, 70, 8000), ((2.6, -2.5, 0.4), 8, 4160, 256),
    ((1.5, -0.5, 0.0), 5, 300, 520),
])
def test_diagonals_are_put_back_where_the_polynomial_adds_a_matrix(co, steps, m, n):
    """b much larger than c, or c zero: A is the addend, and its diagonal's remainder enters
    the square's as dA + Ad + dd."""
    g = momentum(1, m, n, size=1.0)
    want = iteration(g, steps, co)
    like = off(with_rounded_operands(g[0], steps, co)[None], want)
    assert off(mxq.orthogonalize(g, steps=steps, coefficients=co), want) <= 1.25 * like
