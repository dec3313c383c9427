"""orthogonalize of matrices of any magnitude that fp32 holds.

The norm is right to a few roundings of fp32 whatever the elements' size, so the error
is that of ordinary matrices: a rounding to bf16 (1.7e-3 in the norm of many elements) and,
for sides above 64, the fp16 roundings of five steps' operands without a common sign,
1.26e-3 (four of 2^-12 / sqrt(3), five times, in squares, twice for the iteration's
slope): sqrt(1.7^2 + 1.26^2) = 2.1e-3, held to 2.2e-3.  Sides up to 64 carry pairs of
fp16: the rounding to bf16 alone, held to 2^-9.
"""
import pytest
import torch

import mx_block_quantization_gb300 as mxq
from tests.gpu_util import require_gpu
from tests.test_gpu_orthogonalize import iteration, momentum, off

pytestmark = pytest.mark.gpu


def bound(m, n):
    return 2.0**-9 if min(m, n) <= 64 else 2.2e-3


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    yield
    assert mxq.device_status(clear=True) == 0


SHAPES = [(1, 48, 70, 0), (2, 130, 200, 0), (1, 200, 130, 3), (1, 96, 4145, 0), (1, 640, 2048, 0), (3, 1, 40, 0)]


@pytest.mark.parametrize("batch,m,n,pad", SHAPES)
@pytest.mark.parametrize("kind,size", [
    ("f32", 1e-40), ("f32", 1e-30), ("f32", 1e-23), ("f32", 1e-20), ("f32", 2e-13), ("f32", 2e13), ("f32", 1e20), ("f32", 1e37),
    ("bf16", 1e-36), ("bf16", 1e-23), ("bf16", 1e20), ("bf16", 1e37),
])
def test_magnitudes_whose_squares_leave_the_range(batch, m, n, pad, kind, size):
    # built at 1 and scaled in 64 bits: an fp32 product by 1e-40 is rounded like a cast
    g = momentum(batch, m, n, "f32", pad, size=1.0).double().mul(size).to({"f32": torch.float32, "bf16": torch.bfloat16}[kind])
    got = mxq.orthogonalize(g, eps=0.0)
    assert off(got, iteration(g, eps=0.0)) <= bound(m, n)
    if pad == 0:
        # the same values with gaps between the rows: their norm may be summed in another order
        room = torch.zeros(batch, m, n + 5, dtype=g.dtype, device="cuda")
        room[..., :n] = g
        assert off(mxq.orthogonalize(room[..., :n], eps=0.0), iteration(g, eps=0.0)) <= bound(m, n)


@pytest.mark.parametrize("small,large", [(1e-30, 1.0), (1.0, 1e30), (1e-30, 1e30), (1e-14, 1e14), (1e-40, 1e-12)])
def test_rows_of_different_magnitudes(small, large):
    """The large rows make the norm; the small ones are nothing beside them."""
    g = momentum(1, 90, 5000, size=1.0)[0].double()
    g[:80] *= small
    g[80:] *= large
    g = g.float()
    want = iteration(g[None], eps=0.0)[0]
    got = mxq.orthogonalize(g, eps=0.0)
    assert off(got[None, 80:], want[None, 80:]) <= 2.2e-3
    # the small rows are below 2^-24 of the norm, so that X holds zeros
    assert float(got[:80].double().norm()) <= 2.0**-12 * float(want[80:].norm())


def test_a_stack_of_magnitudes():
    g = momentum(6, 70, 120, size=1.0).double()
    sizes = [1e-38, 1e-25, 1e-10, 1.0, 1e10, 1e30]
    g = torch.stack([x * s for x, s in zip(g, sizes)]).float()
    got = mxq.orthogonalize(g, eps=0.0)
    assert off(got, iteration(g, eps=0.0)) <= 2.2e-3
    for x, y in zip(g, got):
        assert torch.equal(mxq.orthogonalize(x, eps=0.0), y) or off(y[None], iteration(x[None], eps=0.0)) <= 2.2e-3


def test_zero_infinite_and_nan():
    z = torch.zeros(70, 80, device="cuda")
    assert (mxq.orthogonalize(z) == 0).all()
    assert mxq.orthogonalize(z, eps=0.0).isnan().all()
    for value in (float("inf"), float("nan")):
        for rest in (0.0, 1e-30, 1.0, 1e30):
            g = torch.full((70, 80), rest, device="cuda")
            g[3, 4] = value
            assert mxq.orthogonalize(g).isnan().any()


def on_the_gpu(g, eps=1e-7):
    """The iteration in 64 bits, a matrix of the stack at a time, by its gram matrix's side."""
    a, b, c = 3.4445, -4.775, 2.0315
    for x in g:
        x = x.double() if x.shape[0] <= x.shape[1] else x.double().t()
        x = x / (x.norm() + eps)
        s = x @ x.t()
        q = torch.eye(s.shape[0], dtype=torch.float64, device="cuda")
        for _ in range(5):  # q: the product of the steps' polynomials, which commute with s
            t = q @ s @ q.t()
            q = (a * torch.eye(s.shape[0], dtype=torch.float64, device="cuda") + b * t + c * t @ t) @ q
        yield q @ x


@pytest.mark.parametrize("batch,m,n", [(40, 1, 1 << 20), (40, 1 << 20, 1), (40, 3, 1 << 19), (2, 1 << 20, 2), (40, 66, 1 << 19),
                                       (9, 600000, 70), (1, 500, 1 << 20)])
def test_very_long_sums(batch, m, n):
    """A gram matrix's sums over the longer side, with few tiles and with many: their fp32
    additions lose 9e-5 at most, which the iteration magnifies less than five times."""
    gen = torch.Generator(device="cuda").manual_seed(m + n)
    g = torch.empty(batch, m, n, dtype=torch.bfloat16, device="cuda")
    for x in g:
        x.copy_(torch.randn(m, n, generator=gen, device="cuda"))
    got = mxq.orthogonalize(g)
    for y, want in zip(got, on_the_gpu(g)):
        y = y.double() if m <= n else y.double().t()
        assert float((y - want).norm() / want.norm()) <= (2.0**-9 if min(m, n) <= 64 else 2.25e-3)


@pytest.mark.parametrize("m,n", [(1 << 20, 1), (1, 1 << 20)])
def test_stacks_of_the_longest_vectors(m, n):
    """A vector's only singular value is its norm: the result is a multiple of it."""
    g = torch.randn(64, m, n, device="cuda")
    norm = g.double().flatten(1).norm(dim=1)
    s = norm / (norm + 1e-7)
    for _ in range(5):
        s = s * (3.4445 - 4.775 * s**2 + 2.0315 * s**4)
    got = mxq.orthogonalize(g).double()
    want = g.double() * (s / norm)[:, None, None]
    assert float(((got - want).flatten(1).norm(dim=1) / s).max()) <= 2.0**-9
