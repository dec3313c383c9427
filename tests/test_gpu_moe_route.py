"""moe_route and moe_route_backward against their definition in 64 bits.

Tolerances: a probability is ex2 of a rounded difference over a sum.  With d the
largest |logit - row maximum| that is not flushed, its relative error is at most
about 2^-23 (2 d log2(e) + 4) from the exponent and the approximation, and the
sum of E <= 1024 terms and the division add less than 20 such units; the tests
use 2^-23 (4 d + 40).  Gradients are sums of such products, held to the same
relative bound of the row's largest term, plus half a unit of bf16 where they are
rounded to it.
"""
import math

import numpy as np
import pytest
import torch

import mx_block_quantization_gb300 as mxq
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    yield
    assert mxq.device_status(clear=True) == 0


def definition(x, k, mask, renorm):
    """float64 [T, E] -> weights, ids, counts, loss, routed, p."""
    T, E = x.shape
    routed = ~(x == -np.inf).all(1) if mask is None else ~(x == -np.inf).all(1) & mask
    w, ids = np.zeros((T, k)), np.full((T, k), -1)
    p = np.zeros((T, E))
    for t in np.flatnonzero(routed):
        with np.errstate(invalid="ignore", over="ignore"):
            top = np.nanmax(x[t]) if not np.isnan(x[t]).all() else np.nan
            z = np.exp(x[t] - top)
            p[t] = z / z.sum()
        rank = np.where(np.isnan(x[t]), -np.inf, x[t])
        best = [e for e in np.argsort(-rank, kind="stable")[:k] if rank[e] > -np.inf]
        ids[t, :len(best)] = best
        w[t, :len(best)] = p[t, best]
        if renorm and best:
            w[t, :len(best)] = np.exp(x[t, best] - top) / np.exp(x[t, best] - top).sum()
    counts = np.bincount(ids[ids >= 0].ravel(), minlength=E)
    n = int(routed.sum())
    loss = E / (k * n * n) * (counts * p.sum(0)).sum() if n else 0.0
    return w, ids, counts, loss, n, p


def gradient(x, k, mask, renorm, dw, dloss):
    w, ids, counts, _, n, p = definition(x, k, mask, renorm)
    T, E = x.shape
    c = dloss * E * counts / (k * n * n) if n else np.zeros(E)
    dx, size = np.zeros((T, E)), np.zeros((T, 1))
    for t in range(T):
        if not p[t].any():
            continue
        live = ids[t] >= 0
        dx[t] = p[t] * (c - (p[t] * c).sum())
        if renorm:
            dx[t, ids[t, live]] += w[t, live] * (dw[t, live] - (w[t, live] * dw[t, live]).sum())
        else:
            g = np.zeros(E)
            g[ids[t, live]] = dw[t, live]
            dx[t] += p[t] * (g - (p[t] * g).sum())
        size[t] = np.abs(c).max() + np.abs(dw[t]).max()
    return dx, size


def bound(x):
    d = x.max(1, keepdims=True) - x
    d = d[np.isfinite(d) & (d < 88)]
    return 2.0**-23 * (4 * (d.max() if d.size else 0.0) + 40)


def logits(T, E, kind, pad=0, seed=0):
    g = torch.Generator().manual_seed(seed + 1000 * T + E)
    x = torch.randn(T, E + pad, generator=g) * 2 + torch.randn(E + pad, generator=g)
    return x.to(TYPES[kind]).cuda()[:, :E]


def check(x, k, mask=None, renorm=True, dw=None, dloss=0.37):
    x64 = x.double().cpu().numpy()
    m = None if mask is None else mask.cpu().numpy().astype(bool)
    r = mxq.moe_route(x, k, mask=mask, renorm=renorm)
    w, ids, counts, loss, n, _ = definition(x64, k, m, renorm)
    tol = bound(x64)
    assert np.array_equal(r.ids.cpu().numpy(), ids)
    assert np.array_equal(r.counts.cpu().numpy(), counts)
    assert int(r.routed) == n
    np.testing.assert_allclose(r.weights.double().cpu().numpy(), w, rtol=tol, atol=1e-37)
    assert float(r.loss) == pytest.approx(loss, rel=tol)
    if dw is None:
        dw = torch.randn(x.shape[0], k, generator=torch.Generator().manual_seed(k)).cuda()
    got = mxq.moe_route_backward(x, r, dw, torch.tensor(dloss, device="cuda"), mask=mask, renorm=renorm)
    assert got.dtype == x.dtype and got.shape == x.shape
    want, size = gradient(x64, k, m, renorm, dw.double().cpu().numpy(), dloss)
    half_unit = 2.0**-8 * np.abs(want) if x.dtype == torch.bfloat16 else 0.0
    assert (np.abs(got.double().cpu().numpy() - want) <= 4 * tol * size + half_unit + 1e-37).all()
    return r, got


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("T,E,k,pad", [
    (1, 1, 1, 0), (1, 64, 8, 0), (2, 2, 1, 1), (33, 3, 3, 0), (31, 8, 2, 0), (5, 60, 4, 4), (40, 63, 6, 1),
    (257, 64, 8, 0), (7, 65, 1, 0), (9, 128, 8, 0), (100, 130, 2, 2), (65, 250, 6, 6), (12, 256, 32, 0),
    (6, 257, 9, 3), (11, 511, 8, 1), (10, 512, 4, 0), (13, 700, 16, 0), (3, 1023, 32, 5), (4, 1024, 8, 0),
])
@pytest.mark.parametrize("renorm", [False, True])
def test_sizes(T, E, k, pad, kind, renorm):
    check(logits(T, E, kind, pad), k, renorm=renorm)


@pytest.mark.parametrize("T,E,k,kind", [(7168, 64, 8, "bf16"), (20011, 250, 6, "f32"), (3001, 384, 3, "bf16")])
def test_many_tokens_use_every_block(T, E, k, kind):
    mask = torch.rand(T, generator=torch.Generator().manual_seed(1)).cuda() > 0.2
    check(logits(T, E, kind), k, mask=mask, renorm=False)


def test_masks_and_rows_without_experts():
    x = logits(50, 20, "f32")
    mask = torch.ones(50, dtype=torch.uint8, device="cuda")
    mask[::3] = 0
    x[7] = -math.inf                    # no expert at all
    x[10, 3:] = -math.inf               # three experts for k = 5
    x[11, :] = torch.finfo(torch.float32).min  # the type's lowest value is a value
    x[13, :19] = torch.finfo(torch.float32).min
    r, dx = check(x, 5, mask=mask)
    assert (r.ids[7] == -1).all() and (r.weights[7] == 0).all() and (dx[7] == 0).all()
    assert r.ids[10].tolist()[3:] == [-1, -1] and r.weights[10, 3:].tolist() == [0, 0]
    assert r.ids[11].tolist() == [0, 1, 2, 3, 4]
    assert (dx[::3] == 0).all()
    check(x, 5, mask=mask.bool(), renorm=False)


def test_every_token_left_out():
    x = logits(9, 16, "bf16")
    r, dx = check(x, 2, mask=torch.zeros(9, dtype=torch.bool, device="cuda"))
    assert float(r.loss) == 0 and int(r.counts.sum()) == 0 and int(r.routed) == 0


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_ties_go_to_the_lowest_index(kind):
    x = torch.randint(-2, 3, (200, 100), generator=torch.Generator().manual_seed(3)).to(TYPES[kind]).cuda()
    x[:, ::7] *= -0.0  # zeros of both signs are equal
    check(x, 8)
    check(torch.zeros(3, 1024, dtype=TYPES[kind], device="cuda"), 32, renorm=False)


def test_nan_and_infinity_stay_in_their_rows_weights():
    x = logits(6, 33, "f32")
    clean = x.clone()
    x[1, 5] = math.nan
    x[2, 0] = math.inf
    x[4] = math.nan
    r = mxq.moe_route(x, 3)
    c = mxq.moe_route(clean, 3)
    for t in (0, 3, 5):
        assert torch.equal(r.ids[t], c.ids[t]) and torch.equal(r.weights[t], c.weights[t])
    assert ((r.ids >= -1) & (r.ids < 33)).all() and 5 not in r.ids[1].tolist() and (r.ids[4] == -1).all()
    assert r.weights[1].isnan().all() and r.weights[2].isnan().all()
    assert math.isnan(float(r.loss)) and int(r.routed) == 6
    dx = mxq.moe_route_backward(x, r, torch.ones_like(r.weights), None)
    want = mxq.moe_route_backward(clean, c, torch.ones_like(r.weights), None)
    assert dx[1].isnan().all() and dx[4].isnan().all()
    for t in (0, 3, 5):
        assert torch.equal(dx[t], want[t])


@pytest.mark.parametrize("renorm", [False, True])
def test_gradient_against_differences(renorm):
    """Central differences of the definition in 64 bits; the choice of experts
    does not change within the step."""
    T, E, k, h = 6, 9, 3, 1e-5
    x = logits(T, E, "f32")
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(8)).cuda()
    r = mxq.moe_route(x, k, renorm=renorm)
    got = mxq.moe_route_backward(x, r, dw, torch.tensor(2.5, device="cuda"), renorm=renorm).double().cpu().numpy()
    x64, g = x.double().cpu().numpy(), dw.double().cpu().numpy()

    def value(v):
        w, _, _, loss, _, _ = definition(v, k, None, renorm)
        return (w * g).sum() + 2.5 * loss
    for t in range(T):
        for e in range(E):
            a, b = x64.copy(), x64.copy()
            a[t, e] += h
            b[t, e] -= h
            assert got[t, e] == pytest.approx((value(a) - value(b)) / (2 * h), abs=2e-5)


def test_either_gradient_alone():
    x = logits(40, 48, "f32")
    r = mxq.moe_route(x, 4, renorm=False)
    dw = torch.randn(40, 4, generator=torch.Generator().manual_seed(5)).cuda()
    dl = torch.tensor(0.5, device="cuda")
    both = mxq.moe_route_backward(x, r, dw, dl, renorm=False)
    one, two = mxq.moe_route_backward(x, r, dw, renorm=False), mxq.moe_route_backward(x, r, None, dl, renorm=False)
    torch.testing.assert_close(both, one + two, rtol=0, atol=2e-6)


def test_no_tokens():
    r = mxq.moe_route(torch.empty(0, 8, device="cuda"), 2)
    assert r.weights.shape == (0, 2) and r.counts.tolist() == [0] * 8 and float(r.loss) == 0 and int(r.routed) == 0
    assert mxq.moe_route_backward(torch.empty(0, 8, device="cuda"), r).shape == (0, 8)


def test_same_bits_every_time_and_on_another_stream():
    x = logits(9001, 96, "f32")
    a = mxq.moe_route(x, 6)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = mxq.moe_route(x, 6, stream=side)
    side.synchronize()
    c = mxq.moe_route(x, 6)
    for f in a._fields:
        assert torch.equal(getattr(a, f), getattr(b, f)) and torch.equal(getattr(a, f), getattr(c, f)), f


def test_captured_into_a_graph():
    x = logits(300, 64, "bf16")
    dl = torch.tensor(0.1, device="cuda")
    warm = mxq.moe_route(x, 4)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r = mxq.moe_route(x, 4)
        dx = mxq.moe_route_backward(x, r, r.weights, dl)
    x.copy_(logits(300, 64, "bf16", seed=9))
    g.replay()
    torch.cuda.synchronize()
    want = mxq.moe_route(x, 4)
    assert not torch.equal(want.ids, warm.ids)
    for f in want._fields:
        assert torch.equal(getattr(r, f), getattr(want, f))
    assert torch.equal(dx, mxq.moe_route_backward(x, want, want.weights, dl))


def test_writes_strided_gradients_and_given_outputs():
    x = logits(37, 50, "bf16", pad=14)
    r = mxq.moe_route(x, 3)
    given = mxq.Routing(*(torch.full_like(t, 7) for t in r))
    assert mxq.moe_route(x, 3, out=given) is given
    for f in r._fields:
        assert torch.equal(getattr(r, f), getattr(given, f))
    wide = torch.full((37, 61), 3.0, dtype=torch.bfloat16, device="cuda")
    mxq.moe_route_backward(x, r, r.weights, r.loss, out=wide[:, :50])
    assert torch.equal(wide[:, :50], mxq.moe_route_backward(x, r, r.weights, r.loss))
    assert (wide[:, 50:] == 3).all()


def test_refusals():
    x = logits(4, 8, "f32")
    for k in (0, 9, -1):
        with pytest.raises((mxq.MxqError, RuntimeError)):
            mxq.moe_route(x, k)
    with pytest.raises(mxq.MxqError):
        mxq.moe_route(logits(2, 40, "f32"), 33)
    with pytest.raises(mxq.MxqError):
        mxq.moe_route(torch.zeros(2, 1025, device="cuda"), 2)
    for bad in (x.cpu(), x.half(), x[0], x.t(), x.double()):
        with pytest.raises(ValueError):
            mxq.moe_route(bad, 2)
    with pytest.raises(ValueError):
        mxq.moe_route(x, 2, mask=torch.ones(5, dtype=torch.bool, device="cuda"))
    with pytest.raises(ValueError):
        mxq.moe_route(x, 2, mask=torch.ones(4, device="cuda"))
    r = mxq.moe_route(x, 2)
    with pytest.raises(ValueError):
        mxq.moe_route_backward(x, r, torch.zeros(4, 3, device="cuda"))
    with pytest.raises(ValueError):
        mxq.moe_route_backward(x, r, r.weights, torch.zeros(1, device="cuda"))
    with pytest.raises(mxq.MxqError) as e:
        mxq.moe_route_backward(x, r, r.weights, out=x)
    assert e.value.code == mxq.EOVERLAP
