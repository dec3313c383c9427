"""orthogonalize against the iteration in 64 bits.

The result is rounded to bf16: a relative error of at most 2^-9, about 2^-9/sqrt(3)
= 1.1e-3 (at most 2e-3) in the Frobenius norm.  Each of the four fp16 operands of a
step (X, A, A', P) adds a relative rounding of at most 2^-12, 2^-12/sqrt(3) = 1.4e-4
in the norm; added up over five steps without cancelling that is 2.8e-3.  The
tests hold the sum, 4.8e-3, for matrices whose singular values stay above the
rounding (random ones, with strong directions over a noise floor).
"""
import numpy as np
import pytest
import torch

import mx_block_quantization_gb300 as mxq
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
COEFFICIENTS = (3.4445, -4.775, 2.0315)
BOUND = 4.8e-3


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    yield
    assert mxq.device_status(clear=True) == 0


def momentum(batch, m, n, kind="f32", pad=0, seed=0, size=1e-3):
    g = torch.Generator().manual_seed(seed + 10000 * m + n)
    few = max(1, min(m, n) // 16)
    x = torch.randn(batch, m, few, generator=g) @ torch.randn(batch, few, n + pad, generator=g) / few**0.5
    return ((x + torch.randn(batch, m, n + pad, generator=g)) * size).to(TYPES[kind]).cuda()[..., :n]


def iteration(g, steps=5, coefficients=COEFFICIENTS, eps=1e-7):
    a, b, c = coefficients
    x = g.double().cpu()
    x = x / (x.flatten(-2).norm(dim=-1)[..., None, None] + eps)
    for _ in range(steps):
        s = x @ x.mT if x.shape[-2] <= x.shape[-1] else x.mT @ x
        p = a * torch.eye(s.shape[-1], dtype=torch.float64) + b * s + c * s @ s
        x = p @ x if x.shape[-2] <= x.shape[-1] else x @ p
    return x


def off(got, want):
    """Largest relative Frobenius error over the stack."""
    d = (got.double().cpu() - want).flatten(-2).norm(dim=-1) / want.flatten(-2).norm(dim=-1)
    return float(d.max())


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("batch,m,n,pad", [
    (1, 64, 64, 0), (1, 128, 256, 0), (1, 256, 128, 0), (1, 256, 256, 0), (2, 200, 333, 0), (1, 333, 200, 3),
    (3, 16, 1000, 0), (2, 1000, 17, 0), (1, 257, 511, 5), (1, 520, 264, 8), (5, 70, 50, 6), (1, 700, 1300, 0),
    (1, 1301, 703, 0), (40, 96, 160, 0), (2, 512, 2048, 0), (1, 2000, 640, 0),
])
def test_sizes(batch, m, n, pad, kind):
    g = momentum(batch, m, n, kind, pad)
    got = mxq.orthogonalize(g)
    assert got.shape == g.shape and got.dtype == torch.bfloat16
    assert off(got, iteration(g)) <= BOUND
    if batch == 1:
        assert torch.equal(mxq.orthogonalize(g[0]), got[0])


@pytest.mark.parametrize("m,n", [(1, 1), (1, 7), (9, 1), (2, 3), (8, 8), (31, 5), (1, 3000), (513, 2)])
def test_smallest_sides(m, n):
    g = momentum(1, m, n)[0] + 1e-4
    assert off(mxq.orthogonalize(g), iteration(g)) <= BOUND


@pytest.mark.parametrize("steps", [1, 2, 3, 8])
def test_steps_and_scale(steps):
    g = momentum(2, 150, 260)
    got = mxq.orthogonalize(g, steps=steps, scale=0.25)
    assert off(got, 0.25 * iteration(g, steps)) <= BOUND * max(1, steps / 5)


def test_other_coefficients():
    g = momentum(1, 180, 140)
    for co in ((1.5, -0.5, 0.0), (15 / 8, -10 / 8, 3 / 8), (2.0, -1.5, 0.5)):
        assert off(mxq.orthogonalize(g, coefficients=co), iteration(g, coefficients=co)) <= BOUND


@pytest.mark.parametrize("size", [1e-12, 1e-6, 1.0, 1e6, 1e12])
def test_any_magnitude(size):
    """The sum of squares stays inside fp32's range."""
    g = momentum(1, 130, 200, size=size)
    assert off(mxq.orthogonalize(g, eps=0.0), iteration(g, eps=0.0)) <= BOUND


def test_singular_values_near_one():
    g = momentum(1, 300, 400)[0]
    s = torch.linalg.svdvals(mxq.orthogonalize(g).double().cpu())
    assert 0.6 < float(s.min()) and float(s.max()) < 1.25


def test_symmetric_in_the_side():
    """The transposed matrix gives the transposed result, to rounding."""
    g = momentum(1, 300, 500)[0]
    a, b = mxq.orthogonalize(g), mxq.orthogonalize(g.t().contiguous())
    assert off(b.t()[None], a.double().cpu()[None]) <= 2 * BOUND


def test_zero_and_not_finite_matrices_stay_by_themselves():
    g = momentum(4, 140, 270)
    clean = mxq.orthogonalize(g)
    g[1] = 0
    g[2, 3, 4] = float("nan")
    got = mxq.orthogonalize(g)
    assert (got[1] == 0).all() and got[2].isnan().any()
    assert torch.equal(got[0], clean[0]) and torch.equal(got[3], clean[3])


def test_strided_output_streams_and_same_bits():
    g = momentum(3, 120, 200, "bf16", pad=8)
    a = mxq.orthogonalize(g)
    assert torch.equal(a, mxq.orthogonalize(g))
    for extra in (8, 3):
        wide = torch.full((3, 125, 200 + extra), 5.0, dtype=torch.bfloat16, device="cuda")
        mxq.orthogonalize(g, out=wide[:, :120, :200])
        assert torch.equal(wide[:, :120, :200], a)
        assert (wide[:, 120:] == 5).all() and (wide[..., 200:] == 5).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = mxq.orthogonalize(g, stream=side)
    side.synchronize()
    assert torch.equal(a, b)


def test_captured_into_a_graph():
    g = momentum(1, 300, 260)[0]
    mxq.orthogonalize(g)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = mxq.orthogonalize(g)
    g.copy_(momentum(1, 300, 260, seed=5)[0])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, mxq.orthogonalize(g))


def test_empty_and_refusals():
    for shape in ((0, 4), (4, 0), (0, 4, 4), (2, 0, 3)):
        assert mxq.orthogonalize(torch.empty(shape, device="cuda")).shape == shape
    g = momentum(1, 20, 30)[0]
    for bad in (g.cpu(), g.half(), g.t(), g[0], g.expand(2, 20, 30)):
        with pytest.raises(ValueError):
            mxq.orthogonalize(bad)
    with pytest.raises(ValueError):
        mxq.orthogonalize(g, out=torch.empty(20, 30, device="cuda"))
    for kw in (dict(steps=0), dict(steps=65), dict(eps=-1.0), dict(eps=float("nan")), dict(scale=float("inf")),
               dict(coefficients=(1.0, float("nan"), 0.0))):
        with pytest.raises(mxq.MxqError):
            mxq.orthogonalize(g, **kw)
    h = momentum(1, 20, 30, "bf16")[0]
    with pytest.raises(mxq.MxqError) as e:
        mxq.orthogonalize(h, out=h)
    assert e.value.code == mxq.EOVERLAP
