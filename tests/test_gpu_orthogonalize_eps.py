"""orthogonalize of matrices far smaller than eps: X = g / (|g| + eps) starts far below 1.

Elementwise the roundings are those of any matrix (fp16's are relative where X keeps out
of its subnormal range), so the bounds are too: 2^-9 for sides up to 64 (bf16's 1.7e-3), and with
four fp16 operands of five steps sqrt(1.7^2 + 1.26^2) = 2.1e-3, held to 2.2e-3.

Through 64 steps, of which up to 50 are linear ones at first, the roundings of X add up:
the coefficients (15/8, -10/8, 3/8) draw singular values together but leave rotated
directions as they are.  Those runs are held to the error of the iteration in 64 bits
whose X is rounded to fp16's 11 bits after each step and to bf16's 8 at the end, and a
quarter more for the other operands and another sample of roundings.
"""
import pytest
import torch

import mx_block_quantization_gb300 as mxq
from tests.gpu_util import require_gpu
from tests.test_gpu_orthogonalize import iteration, momentum, off

pytestmark = pytest.mark.gpu
CONTRACTING = (15 / 8, -10 / 8, 3 / 8)


def bound(m, n):
    return 2.0**-9 if min(m, n) <= 64 else 2.2e-3


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    yield
    assert mxq.device_status(clear=True) == 0


def of_norm(g, norm):
    """Each matrix of the stack scaled to this Frobenius norm, in fp32."""
    g = g.double()
    return (g * (norm / g.flatten(-2).norm(dim=-1)[..., None, None])).float()


@pytest.mark.parametrize("batch,m,n,pad", [
    (1, 48, 70, 0), (2, 130, 200, 0), (1, 200, 130, 3), (1, 96, 4145, 0), (1, 40, 9000, 0), (1, 640, 2048, 0), (1, 1500, 300, 0),
])
@pytest.mark.parametrize("norm,eps", [(1e-14, 1e-7), (1e-17, 1e-7), (1e-10, 1e-7), (6e-8, 1e-7), (1e-7, 1e-7), (1e-30, 1e-7),
                                      (1.0, 1e6), (1e-20, 1.0)])
def test_far_below_eps(batch, m, n, pad, norm, eps):
    g = of_norm(momentum(batch, m, n, pad=pad, size=1.0), norm)
    got, want = mxq.orthogonalize(g, eps=eps), iteration(g, eps=eps)
    assert off(got, want) <= bound(m, n)
    assert torch.equal(got, mxq.orthogonalize(g, eps=eps))


@pytest.mark.parametrize("batch,m,n", [(1, 50, 60), (1, 130, 200), (1, 260, 140), (1, 72, 5000)])
@pytest.mark.parametrize("norm", [1e-8, 1e-11, 1e-14])
@pytest.mark.parametrize("steps", [1, 2, 7])
def test_from_far_below_to_one(batch, m, n, norm, steps):
    g = of_norm(momentum(batch, m, n, size=1.0), norm)
    got = mxq.orthogonalize(g, steps=steps, coefficients=CONTRACTING)
    assert off(got, iteration(g, steps, CONTRACTING)) <= bound(m, n)


def with_rounded_x(g, steps, coefficients, eps=1e-7):
    a, b, c = coefficients

    def rounded(x, bits):
        f, e = torch.frexp(x)
        return torch.ldexp(torch.round(f * 2.0**bits), e - bits)

    x = g.double().cpu()
    x = rounded(x / (x.norm() + eps), 11)
    for s in range(steps):
        q = x @ x.mT if x.shape[0] <= x.shape[1] else x.mT @ x
        p = a * torch.eye(q.shape[0], dtype=torch.float64) + b * q + c * q @ q
        x = rounded(p @ x if x.shape[0] <= x.shape[1] else x @ p, 11 if s + 1 < steps else 8)
    return x


@pytest.mark.parametrize("m,n", [(50, 60), (130, 200), (260, 140), (72, 5000)])
@pytest.mark.parametrize("norm", [1.0, 1e-8, 1e-11, 1e-14])
def test_many_steps_from_far_below_to_one(m, n, norm):
    g = of_norm(momentum(1, m, n, size=1.0), norm)
    want = iteration(g, 64, CONTRACTING)
    like = off(with_rounded_x(g[0], 64, CONTRACTING)[None], want)
    got = off(mxq.orthogonalize(g, steps=64, coefficients=CONTRACTING), want)
    assert got <= (2.0**-9 if min(m, n) <= 64 else 1.25 * like)


def test_other_forms_of_the_polynomial():
    """c zero and b much larger than c (the addend from memory), and a below 1."""
    g = of_norm(momentum(2, 150, 210, size=1.0), 1e-13)
    for co in ((1.5, -0.5, 0.0), (1.6, -0.65, 0.05), (0.9, 0.05, 0.0)):
        assert off(mxq.orthogonalize(g, coefficients=co), iteration(g, coefficients=co)) <= 2.2e-3


def test_each_matrix_of_a_stack_by_itself():
    norms = [1e-25, 1e-14, 1e-9, 1e-7, 1e-3, 1.0, 0.0]
    g = torch.stack([of_norm(x, s) for x, s in zip(momentum(7, 130, 90, size=1.0), norms)])
    got, want = mxq.orthogonalize(g), iteration(g)
    assert (got[6] == 0).all() and off(got[:6], want[:6]) <= 2.2e-3
    for x, y in zip(g, got):
        assert torch.equal(mxq.orthogonalize(x), y) or off(y[None], iteration(x[None])) <= 2.2e-3


def test_scale_and_both_kinds_of_output():
    g = of_norm(momentum(1, 140, 99, size=1.0), 1e-15)[0]
    want = 3e4 * iteration(g[None])[0]
    for out in (None, torch.empty(140, 101, dtype=torch.bfloat16, device="cuda")[:, :99]):
        got = mxq.orthogonalize(g, scale=3e4, out=out)
        assert off(got[None], want[None]) <= 2.2e-3


def test_results_below_the_normal_numbers_end_in_zero():
    """|g| / eps of 1e-42: the result is below bf16's range, not NaN."""
    g = of_norm(momentum(1, 80, 90, size=1.0), 1e-30)
    got = mxq.orthogonalize(g, eps=1e12)
    assert got.isfinite().all() and float(got.abs().max()) < 1e-36
