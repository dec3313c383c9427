"""moe_route_groups and its gradient against their definition in 64 bits.

The choice has to be the definition's, whatever the rounding.  Tolerances of the rest: a
score is a reciprocal of one plus an exponential, or an exponential over a sum.  With d
the largest |logit| (or distance from the row's largest) whose exponential is not flushed,
its relative error is at most about 2^-23 (2 d log2(e) + 4) from the exponent and the
approximations; sums of E <= 1024 terms and the divisions add less than 20 such units:
2^-23 (4 d + 40), as in the tests of moe_route.  The largest d of values that matter in
fp32 is 88.  Gradients are sums of such products and are held to the same bound of the
row's largest term, plus half a unit of bf16 where they are rounded to it.
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
    torch.cuda.empty_cache()
    assert mxq.device_status(clear=True) == 0


def scores_of(x, kind):
    with np.errstate(invalid="ignore", over="ignore"):
        if kind == "sigmoid":
            return 1 / (1 + np.exp(-x))
        top = np.fmax.reduce(x, axis=1, keepdims=True)
        z = np.exp(x - top)
        return z / z.sum(1, keepdims=True)


def choose(s, x, bias, k, groups, best):
    """The chosen experts of each row, -1 where there are no more."""
    T, E = x.shape
    c = s + bias
    c = np.where((x > -np.inf) & (c > -np.inf), c, -np.inf)      # not NaN
    ids = np.full((T, k), -1)
    for t in range(T):
        v = c[t].copy()
        if best < groups:
            size, value = E // groups, []
            for g in range(groups):
                two = [a for a in np.sort(v[g * size:(g + 1) * size])[::-1][:2] if a > -np.inf]
                value.append(sum(two) if two else -np.inf)
            kept = np.argsort(-np.array(value), kind="stable")[:best]
            for g in set(range(groups)) - set(kept.tolist()):
                v[g * size:(g + 1) * size] = -np.inf
        order = [e for e in np.argsort(-v, kind="stable")[:k] if v[e] > -np.inf]
        ids[t, :len(order)] = order
    return ids


class Case:
    def __init__(self, T, E, k, groups=1, best=1, scores="sigmoid", kind="f32", pad=0, seed=0, bias="some", x=None):
        g = torch.Generator().manual_seed(seed + 1000 * T + E)
        if x is None:
            x = torch.randn(T, E + pad, generator=g) * 2 + torch.randn(E + pad, generator=g)
        self.x = x.to(TYPES[kind]).cuda()[:, :E]
        self.bias = {"some": torch.randn(E, generator=g) * 0.1, "zero": torch.zeros(E), "none": None,
                     "few": torch.randint(-2, 3, (E,), generator=g) * 0.001}[bias] if isinstance(bias, str) else bias
        self.bias = None if self.bias is None else self.bias.cuda()
        self.k, self.how = k, dict(scores=scores)
        self.groups = dict(groups=groups, best_groups=best)

    def check(self, mask=None, renorm=True, scale=1.0, dloss=0.37, exact=True):
        x, k, how = self.x.double().cpu().numpy(), self.k, self.how
        T, E = x.shape
        m = np.ones(T, bool) if mask is None else mask.cpu().numpy().astype(bool)
        routed = m & ((x > -np.inf) | np.isnan(x)).any(1)
        b = np.zeros(E) if self.bias is None else self.bias.double().cpu().numpy()
        s = scores_of(x, how["scores"])
        ids = choose(s, x, b, k, self.groups["groups"], self.groups["best_groups"])
        ids[~routed] = -1
        r = mxq.moe_route_groups(self.x, k, bias=self.bias, mask=mask, renorm=renorm, scale=scale, **how, **self.groups)
        assert np.array_equal(r.ids.cpu().numpy(), ids)
        assert np.array_equal(r.counts.cpu().numpy(), np.bincount(ids[ids >= 0].ravel(), minlength=E))
        assert int(r.routed) == routed.sum()
        if not exact:
            return r
        d = np.abs(x) if how["scores"] == "sigmoid" else np.fmax.reduce(x, axis=1, keepdims=True) - x
        d = d[np.isfinite(d) & (d < 88)]
        tol = 2.0**-23 * (4 * (d.max() if d.size else 0.0) + 40)
        live = ids >= 0
        picked = np.where(live, np.take_along_axis(s, np.maximum(ids, 0), 1), 0.0)
        total = picked.sum(1, keepdims=True) if renorm else np.ones((T, 1))
        w = np.where(total > 0, picked / np.where(total > 0, total, 1), 0.0)
        np.testing.assert_allclose(r.weights.double().cpu().numpy(), scale * w, rtol=tol, atol=1e-37)
        n, counts = int(routed.sum()), np.bincount(ids[live].ravel(), minlength=E)
        every = np.where(routed[:, None], s, 0).sum(1, keepdims=True)
        p = np.where(routed[:, None] & (every > 0), s / np.where(every > 0, every, 1), 0.0)
        loss = E / (k * n * n) * (counts * p.sum(0)).sum() if n else 0.0
        assert float(r.loss) == pytest.approx(loss, rel=tol)
        # gradient
        dw = torch.randn(T, k, generator=torch.Generator().manual_seed(k)).cuda()
        got = mxq.moe_route_groups_backward(self.x, r, dw, torch.tensor(dloss, device="cuda"), mask=mask, renorm=renorm,
                                            scale=scale, **how)
        dwn = np.where(live, dw.double().cpu().numpy() * scale, 0.0)
        part = (dwn - (w * dwn).sum(1, keepdims=True)) / np.where(total > 0, total, np.inf) if renorm else dwn
        g = np.zeros((T, E))
        for t in range(T):
            g[t, ids[t][live[t]]] = part[t][live[t]]
        c = dloss * E * counts / (k * n * n) if n else np.zeros(E)
        size = np.abs(part).max(1, keepdims=True) + np.abs(dwn).max(1, keepdims=True) / np.where(total > 0, total, np.inf)
        if how["scores"] == "sigmoid":
            slope = np.where(np.isfinite(x), 1 / (2 + np.exp(np.minimum(np.abs(x), 700)) + np.exp(-np.abs(x))), 0.0)
            back = np.where(every > 0, 1 / np.where(every > 0, every, 1), 0.0)
            want = slope * (g + (c - (p * c).sum(1, keepdims=True)) * back)
            bound = slope * (size + 2 * np.abs(c).max() * back)
        else:
            h = g + c
            want = p * (h - (p * h).sum(1, keepdims=True))
            bound = p * 2 * (size + np.abs(c).max())
        want[~routed] = 0
        off = 4 * tol * bound + (2.0**-8 * np.abs(want) if self.x.dtype == torch.bfloat16 else 0) + 1e-37
        assert (np.abs(got.double().cpu().numpy() - want) <= off).all()
        assert got.dtype == self.x.dtype and got.shape == self.x.shape
        return r


SIZES = [(1, 1, 1, 1, 1, 0), (1, 64, 8, 8, 4, 0), (3, 6, 2, 3, 2, 1), (33, 30, 3, 6, 1, 0), (31, 32, 8, 32, 9, 0), (5, 60, 4, 4, 3, 4),
         (40, 64, 6, 8, 3, 1), (257, 64, 8, 1, 1, 0), (9, 128, 8, 2, 1, 0), (100, 130, 2, 26, 5, 2), (65, 250, 6, 5, 2, 6),
         (12, 256, 32, 8, 4, 0), (50, 256, 8, 8, 4, 0), (6, 260, 9, 20, 7, 3), (11, 511, 8, 7, 3, 1), (10, 512, 4, 32, 8, 0),
         (13, 700, 16, 10, 10, 0), (3, 1023, 32, 31, 2, 5), (4, 1024, 8, 32, 1, 0), (20, 96, 20, 3, 1, 0)]


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("scores", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,k,groups,best,pad", SIZES)
def test_sizes(T, E, k, groups, best, pad, scores, kind):
    case = Case(T, E, k, groups, best, scores, kind, pad)
    case.check(renorm=False, scale=2.5)
    case.check()


@pytest.mark.parametrize("scores", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,k,groups,best,kind", [(7168, 64, 6, 8, 4, "bf16"), (5003, 250, 6, 5, 3, "f32"), (3001, 384, 3, 1, 1, "bf16")])
def test_many_tokens_use_every_block(T, E, k, groups, best, kind, scores):
    mask = torch.rand(T, generator=torch.Generator().manual_seed(1)).cuda() > 0.2
    case = Case(T, E, k, groups, best, scores, kind)
    first, again = case.check(mask), case.check(mask.to(torch.uint8))
    for a, b in zip(first, again):
        assert torch.equal(a, b)


@pytest.mark.parametrize("scores", ["sigmoid", "softmax"])
@pytest.mark.parametrize("bias", ["none", "zero", "few", "some"])
@pytest.mark.parametrize("groups,best", [(1, 1), (8, 4), (8, 1)])
def test_equal_logits_and_near_ones(groups, best, bias, scores):
    """bf16 logits of few values; values one unit in the last place apart; all alike."""
    g = torch.Generator().manual_seed(3)
    few = torch.randint(-3, 4, (60, 128), generator=g) * 0.5
    Case(60, 128, 6, groups, best, scores, "bf16", bias=bias, x=few).check()
    Case(60, 128, 16, groups, best, scores, "f32", bias=bias, x=torch.full((60, 128), 0.25)).check()
    near = torch.full((60, 128), 1.0) + torch.randint(0, 8, (60, 128), generator=g) * 2.0**-23
    Case(60, 128, 6, groups, best, scores, "f32", bias=bias, x=near).check()


def test_scores_nearer_than_fp32_can_tell():
    """Logits whose scores are one in fp32, told apart by 64 bits; and a bias that crosses them."""
    g = torch.Generator().manual_seed(4)
    high = torch.randint(0, 1000, (40, 96), generator=g) * 0.01 + 18.0
    low = -high - 20.0
    for x in (high, low):
        for bias in ("none", "zero", "few"):
            Case(40, 96, 7, 6, 2, "sigmoid", "f32", bias=bias, x=x).check(exact=False)
            Case(40, 96, 7, 1, 1, "sigmoid", "f32", bias=bias, x=x).check(exact=False)
    # s + bias equal to within 2^-26: the sum of logistic(x) and what is left of one
    x = torch.randn(200, 64, generator=g)
    bias = torch.zeros(64)
    s = torch.sigmoid(x[0].double())
    bias = (1.0 - s).float()
    x[:] = x[0]
    Case(200, 64, 8, 8, 3, "sigmoid", "f32", bias=bias, x=x).check()
    s = torch.softmax(x[0].double(), 0)
    Case(200, 64, 8, 8, 3, "softmax", "f32", bias=(0.1 - s).float(), x=x).check()


@pytest.mark.parametrize("scores", ["sigmoid", "softmax"])
def test_experts_that_must_not_be_chosen(scores):
    """Logits of -inf, biases of -inf; rows, groups and choices that stay empty."""
    x = torch.randn(50, 48, generator=torch.Generator().manual_seed(5))
    x[0] = -math.inf
    x[1, 1:] = -math.inf
    x[2, :24] = -math.inf
    x[3, 3:] = -math.inf
    x[4:, 8:16] = -math.inf
    bias = torch.zeros(48)
    bias[16:24] = -math.inf
    bias[47] = math.inf
    mask = torch.ones(50, dtype=torch.bool)
    mask[10:20] = False
    for groups, best, k in ((6, 2, 5), (6, 1, 8), (1, 1, 8), (6, 6, 3), (2, 1, 24), (24, 5, 4)):
        for b in ("zero", bias):
            Case(50, 48, k, groups, best, scores, "f32", bias=b, x=x).check(mask.cuda())
    empty = Case(50, 48, 4, 6, 2, scores, "f32", x=x).check(torch.zeros(50, dtype=torch.bool, device="cuda"))
    assert int(empty.routed) == 0 and float(empty.loss) == 0 and bool((empty.ids == -1).all())


def test_values_that_are_not_finite():
    x = torch.randn(6, 32, generator=torch.Generator().manual_seed(6))
    x[0, 3], x[1, 4], x[2, 5] = math.nan, math.inf, math.nan
    x[2, 6:] = math.nan
    case = Case(6, 32, 4, 4, 2, "sigmoid", "f32", bias="some", x=x)
    r = case.check(exact=False)
    assert math.isnan(float(r.loss)) and bool(torch.isfinite(r.weights).all()) and 4 in r.ids[1].tolist()
    r = Case(6, 32, 4, 4, 2, "softmax", "f32", bias="some", x=x).check(exact=False)
    assert bool((r.ids[:3] == -1).all()) and bool((r.ids[3:] >= 0).all())


def test_scores_that_vanish():
    """A row whose scores are zero in fp32: weights of zero, no gradient, no NaN."""
    x = torch.full((4, 16), -200.0)
    x[3] = torch.randn(16)
    r = mxq.moe_route_groups(x.cuda(), 3, groups=4, best_groups=2)
    assert not r.weights[:3].any() and bool((r.ids >= 0).all()) and bool(torch.isfinite(r.loss))
    dx = mxq.moe_route_groups_backward(x.cuda(), r, torch.ones(4, 3, device="cuda"), torch.ones((), device="cuda"))
    assert not dx[:3].any() and bool(torch.isfinite(dx).all())


def test_without_bias_and_groups_softmax_is_moe_route():
    x = Case(300, 200, 6).x
    mask = torch.rand(300, device="cuda") > 0.1
    a, b = mxq.moe_route(x, 6, mask=mask), mxq.moe_route_groups(x, 6, scores="softmax", mask=mask)
    assert torch.equal(a.ids, b.ids) and torch.equal(a.counts, b.counts) and torch.equal(a.routed, b.routed)
    torch.testing.assert_close(a.weights, b.weights, rtol=2.0**-19, atol=0)
    torch.testing.assert_close(a.loss, b.loss, rtol=2.0**-18, atol=0)


@pytest.mark.parametrize("scores", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [False, True])
def test_gradient_by_differences(scores, renorm):
    """Central differences of the fp32 forward call: with steps of h = 2^-6 they are off by
    h^2/6 of third derivatives of at most about 1 and by 2^-22 / h of the rounding."""
    T, E, k, h = 3, 24, 4, 2.0**-6
    case = Case(T, E, k, 4, 2, scores, bias=torch.arange(24) % 4 * 3.0)    # no step changes the choice
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(9)).cuda()
    how = dict(scores=scores, renorm=renorm, scale=1.5)
    r = mxq.moe_route_groups(case.x, k, bias=case.bias, **case.groups, **how)
    got = mxq.moe_route_groups_backward(case.x, r, dw, torch.tensor(2.0, device="cuda"), **how)

    def value(x):
        q = mxq.moe_route_groups(x, k, bias=case.bias, **case.groups, **how)
        assert torch.equal(q.ids, r.ids)
        return float((q.weights.double() * dw.double()).sum() + 2.0 * q.loss.double())

    for t in range(T):
        for e in range(E):
            up, down = case.x.clone(), case.x.clone()
            up[t, e] += h
            down[t, e] -= h
            slope = (value(up) - value(down)) / float(up[t, e].double() - down[t, e].double())
            assert abs(slope - float(got[t, e])) <= 20 * (h * h / 6 + 2.0**-22 / h)


def test_strides_streams_and_replay():
    case = Case(300, 64, 6, 8, 4, pad=3)
    want = case.check()
    how = dict(bias=case.bias, **case.groups)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = mxq.moe_route_groups(case.x, 6, stream=side, **how)
    dw = torch.ones(300, 6, device="cuda")
    room = torch.full((300, 70), 7.0, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    dx = mxq.moe_route_groups_backward(case.x, got, dw, stream=side, out=room[:, 2:66])
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert bool((room[:, :2] == 7).all()) and bool((room[:, 66:] == 7).all())
    assert torch.equal(dx, mxq.moe_route_groups_backward(case.x, want, dw))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = mxq.moe_route_groups(case.x, 6, **how)
        d = mxq.moe_route_groups_backward(case.x, r, dw)
    for seed in range(3):
        case.x.copy_(Case(300, 64, 6, seed=seed).x)
        graph.replay()
        again = mxq.moe_route_groups(case.x, 6, **how)
        assert all(torch.equal(a, b) for a, b in zip(r, again))
        assert torch.equal(d, mxq.moe_route_groups_backward(case.x, again, dw))


def test_no_tokens():
    x = torch.empty(0, 64, device="cuda")
    r = mxq.moe_route_groups(x, 4, groups=8, best_groups=2)
    assert r.ids.shape == (0, 4) and not r.counts.any() and float(r.loss) == 0 and int(r.routed) == 0
    assert mxq.moe_route_groups_backward(x, r, r.weights).shape == (0, 64)


@pytest.mark.parametrize("size", [2, 32])
@pytest.mark.parametrize("scores", ["sigmoid", "softmax"])
def test_large_biases_that_cancel_in_a_group(scores, size):
    """A group's two largest are about +100 and -100 off: what fp32 loses of each is more than its sum's own rounding."""
    E, T = 16 * size, 40000 // size
    bias = torch.full((E,), -100.0)
    bias[::size] = 100.0
    x = torch.randn(T, E, generator=torch.Generator().manual_seed(8))
    Case(T, E, 5, 16, 5, scores, "f32", bias=bias, x=x).check(exact=False)


@pytest.mark.parametrize("T,E,groups,best", [(400, 64, 1, 1), (400, 64, 32, 20), (300, 200, 8, 5), (200, 510, 2, 1)])
@pytest.mark.parametrize("scores", ["sigmoid", "softmax"])
def test_the_most_choices_of_a_token(scores, T, E, groups, best):
    """32 of them, the next ones at some distance, near, and alike."""
    g = torch.Generator().manual_seed(9)
    x = torch.randn(T, E, generator=g)
    Case(T, E, 32, groups, best, scores, "f32", x=x).check()
    Case(T, E, 32, groups, best, scores, "bf16", bias="zero", x=x).check()
    # Two groups with the same two scores and the same two biases, the other way round, have
    # sums that are equal, and in 64 bits differ by their roundings: at most 4 of values
    # below 2, 4 * 2^-53.  Rows whose choice of groups hangs on less are left out.
    few = Case(T, E, 32, groups, best, scores, "f32", bias="few", x=torch.round(2 * x) / 2)
    c = scores_of(few.x.double().cpu().numpy(), scores) + few.bias.double().cpu().numpy()
    value = np.sort(np.sort(c.reshape(T, groups, -1), axis=2)[:, :, -2:].sum(2), axis=1)[:, ::-1]
    if best < groups:
        few.x = few.x[torch.from_numpy(value[:, best - 1] - value[:, best] > 2.0**-51).cuda()]
        assert few.x.shape[0] > T // 2
    few.check()


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("scores", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,groups,best,k", [(64, 8, 4, 6), (64, 64 // 2, 5, 10), (200, 1, 1, 32), (510, 2, 1, 8), (1024, 32, 2, 32)])
def test_rows_of_one_value(E, groups, best, k, scores, kind):
    """Of zeros, of others with one bias for all, and with an expert left out, an infinite one, one that is not a number."""
    x = torch.zeros(12, E)
    x[1], x[2], x[3], x[4] = -3.5, 20.0, -90.0, 0.25
    x[5, 0], x[6, E - 1], x[7, 1], x[8, E // 2] = -torch.inf, -torch.inf, 0.5, -0.0
    x[9] = -torch.inf
    # 1 / (1 + e^90) = 8.2e-40 is below 2^-126 = 1.2e-38, where a score is 0 and so are weights
    # over such scores' sum: the choice is compared for that row, the rest without it
    held = torch.tensor([t for t in range(12) if t != 3 or scores == "softmax"])
    for bias in ("none", torch.full((E,), -0.75)):
        Case(12, E, k, groups, best, scores, kind, bias=bias, x=x).check(exact=False)
        Case(len(held), E, k, groups, best, scores, kind, bias=bias, x=x[held]).check()
    if scores == "sigmoid":  # a row of its own with softmax has no score at all
        x[10], x[11, 3] = torch.inf, torch.nan
        Case(12, E, k, groups, best, scores, kind, bias="zero", x=x).check(exact=False)
    Case(12, E, k, groups, best, scores, kind, bias=torch.full((E,), torch.inf), x=x).check(exact=False)
    Case(12, E, k, groups, best, scores, kind, bias=torch.full((E,), -torch.inf), x=x).check(exact=False)
