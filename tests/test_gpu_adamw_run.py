"""Moments in 8 bits over a run of steps, against those in 32 bits from the same gradients.

A step's bytes are compared elsewhere; this is what many roundings leave.  The root r of v is
rounded at random with itself as mean, so the mean of its square, which is v, gains the
rounding's variance.  With gap G between E4M3 values and a root that moves by d that is at
most G d; d is r (1 - b2) / (1 + sqrt(b2)) |g^2 / v - 1|, G at most r / 8, and |g^2 / v - 1|
0.968 on the mean for normal gradients: (1 - b2) times 0.061 of v a step, of which (1 - b2)
is forgotten in each.  So v lies between 0 and 6.1% too high on the mean, 6.5% with the
deviations of r from sqrt(v) within d, and the mean of 131072 elements, each some 30% off,
is within five deviations, 0.4%, of that.
"""
import pytest
import torch

import mx_block_quantization_gb300 as mxq
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    yield
    torch.cuda.empty_cache()
    assert mxq.device_status(clear=True) == 0


def values(q, s):
    return q.view(torch.float8_e4m3fn).double() * torch.exp2(s.double() - 127).repeat_interleave(32)


def run(gradients, steps, beta2):
    """(parameters, m, v) of both kinds of moments after so many steps."""
    g = gradients(0)
    out = []
    for bits in (8, 32):
        p = torch.zeros_like(g)
        moments = mxq.adamw_moments([p], bits)
        for t in range(1, steps + 1):
            mxq.adamw_step([p], [gradients(t)], moments, t, lr=1e-3, betas=(0.9, beta2), weight_decay=0.0, seed=11)
        if bits == 8:
            out.append((p, values(moments.m, moments.m_scale), values(moments.v, moments.v_scale) ** 2))
        else:
            out.append((p, moments.m.double(), moments.v.double()))
    return out


@pytest.mark.parametrize("beta2,steps", [(0.95, 200), (0.999, 6000)])
def test_v_is_a_little_high_on_the_mean(beta2, steps):
    def gradients(t):
        return torch.randn(131072, generator=torch.Generator(device="cuda").manual_seed(t), device="cuda")

    (p8, m8, v8), (p32, m32, v32) = run(gradients, steps, beta2)
    ratio = float(v8.mean() / v32.mean())
    print(f"beta2 {beta2}: v {ratio:.4f} of the exact one on the mean, single ones {float((v8 / v32).min()):.2f} to {float((v8 / v32).max()):.2f}")
    assert 1 - 0.004 < ratio < 1.065 + 0.004
    # m has no square: a mean of 0, each off by up to a root of (1 + 0.9^2 + ...) / 2 gaps of 2^-3, 7% in the mean of sizes
    assert abs(float((m8 - m32).mean())) < 5 * 0.15 * float(m32.abs().mean()) / 131072**0.5


def test_small_gradients_beside_large_ones():
    """A root is not rounded to 0 but to the smallest value of its block, here 2^-17 for
    gradients of 1e-7 beside one of 1: their steps are 1e-7 / 2^-17 = 1 / 76 of those of
    moments in 32 bits, in jumps, a hundredth of them within a tenth."""
    g = torch.full((32 * 64,), 1e-7, device="cuda")
    g[::32] = 1.0
    (p8, _, v8), (p32, _, v32) = run(lambda t: g, 200, 0.95)
    small = torch.ones(32 * 64, dtype=torch.bool, device="cuda")
    small[::32] = False
    assert bool((v8[small] >= 2.0**-34).all()) and float(v32[small].max()) < 1.1e-14
    assert 0 < float(p8[small].mean() / p32[small].mean()) < 0.1
    assert float((p8[~small] / p32[~small] - 1).abs().max()) < 0.2
