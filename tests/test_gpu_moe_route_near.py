"""moe_route_groups where the choice hangs on less than fp32 can tell, against 64 bits.

The definition's choice is compared bit for bit, so there is no tolerance.  A row is left
out where two values that its choice hangs on lie within 2^-44 in 64 bits: the definition
here and the kernel's own 64-bit pass are each right to some 2^-50 of values below 4.
"""
import numpy as np
import pytest
import torch

import mx_block_quantization_gb300 as mxq
from tests.gpu_util import require_gpu
from tests.test_gpu_moe_route_groups import choose, scores_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    yield
    torch.cuda.empty_cache()
    assert mxq.device_status(clear=True) == 0


def compare(x, bias, k, groups=1, best=1, scores="softmax", keep=None):
    """ids of the rows that `keep` names."""
    wide = x.double().numpy()
    want = choose(scores_of(wide, scores), wide, bias.double().numpy(), k, groups, best)
    got = mxq.moe_route_groups(x.cuda(), k, bias=bias.cuda(), scores=scores, groups=groups, best_groups=best).ids.cpu().numpy()
    keep = np.ones(len(want), bool) if keep is None else keep
    wrong = (got != want).any(1) & keep
    assert not wrong.any(), f"{wrong.sum()} of {keep.sum()} rows, the first: {got[wrong][0]} for {want[wrong][0]}"


# experts in one group: one, two and eight of them a lane, and more than the lanes own
@pytest.mark.parametrize("E", [32, 64, 256, 512])
@pytest.mark.parametrize("at", [0.01, 0.1])
@pytest.mark.parametrize("between", [0, 1])
def test_a_large_score_that_its_bias_takes_back(E, at, between):
    """An expert whose score of about 0.9 loses most of it to its bias, next to one whose
    score is small: what fp32 is off by is the first one's, whichever comes first.  With
    `between` another small one lies next to the second, and the first is two places down."""
    for seed in range(6):
        g = torch.Generator().manual_seed(seed)
        base = -9.0 - 3.0 * torch.rand(E, generator=g)
        first, second, third = torch.randperm(E, generator=g)[:3].tolist()
        base[first], base[second], base[third] = 0.0, -4.0 - 0.5 * seed, -4.25 - 0.5 * seed
        T = 400
        x = base.repeat(T, 1)
        # the large score moves by s (1 - s) 2^-21 from row to row, about 4e-8
        x[:, first] += (torch.arange(T) - T // 2) * 2.0**-21
        s = torch.softmax(base.double(), 0)
        bias = torch.full((E,), -0.3)
        bias[first] = (at - s[first]).float()
        bias[second] = (at - s[second]).float()
        if between:
            bias[third] = (at - 3e-7 - s[third]).float()
        c = torch.softmax(x.double(), 1) + bias.double()
        top = torch.sort(c, 1, descending=True).values[:, :4]
        keep = ((top[:, :-1] - top[:, 1:]) > 2.0**-44).all(1).numpy()
        assert keep.sum() > T // 2
        for k in (1, 2, 3):
            compare(x, bias, k, keep=keep)


LOWEST = torch.finfo(torch.float32).min


@pytest.mark.parametrize("scores", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,groups,best,k", [(32, 4, 2, 10), (64, 4, 3, 20), (256, 8, 2, 32), (288, 8, 2, 32), (512, 32, 2, 20), (1024, 32, 2, 32)])
def test_experts_left_out_by_the_lowest_bias(E, groups, best, k, scores):
    """Groups whose experts all have a bias of the type's lowest value come last, and are
    chosen where no others are left: the sum of two of them leaves fp32's range, not 64
    bits' (the scores vanish in it there too, so equal ones go by their index)."""
    x = torch.randn(30, E, generator=torch.Generator().manual_seed(11))
    size = E // groups
    for live in (1, best, groups):
        bias = torch.zeros(E)
        for group in range(groups):
            if group >= live:
                bias[group * size:(group + 1) * size] = LOWEST
        compare(x, bias, k, groups, best, scores)
        compare(x, bias.flip(0), k, groups, best, scores)
    bias = torch.zeros(E)
    bias[::2] = LOWEST
    compare(x, bias, min(k, size), groups, best, scores)
    compare(x, torch.full((E,), LOWEST), k, groups, best, scores)


@pytest.mark.parametrize("groups,best", [(1, 1), (8, 3)])
@pytest.mark.parametrize("E", [32, 128, 256, 512])
def test_small_scores_near_one_another(E, groups, best):
    """Sigmoid scores of 1e-4 to 1e-11, logits a few units in the last place apart and equal
    ones; without a bias, with one for all and with one that takes the scores' order back."""
    g = torch.Generator().manual_seed(12)
    for shift in (-9.0, -14.0, -19.0, -25.0):
        at = shift - 0.25 * torch.randint(0, 4, (60, E), generator=g)
        x = at + torch.randint(-3, 4, (60, E), generator=g) * 2.0**-20
        s = torch.sigmoid(x[0].double())
        for bias in (torch.zeros(E), torch.full((E,), 0.001), (s.max() - s).float()):
            c = torch.sigmoid(x.double()) + bias.double()
            # two scores and two biases the other way round have sums that are equal but for
            # their roundings, as have groups of such pairs: rows without near sums are kept
            if groups > 1:
                value = torch.topk(c.view(60, groups, -1), 2, dim=2).values.sum(2).sort(1, descending=True).values
                keep = value[:, best - 1] - value[:, best] > 2.0**-50 * value[:, 0].abs()
            else:
                keep = torch.ones(60, dtype=torch.bool)
            compare(x, bias, 8, groups, best, "sigmoid", keep.numpy())


def choose_all(x, bias, k, groups, best, scores):
    """ids of all rows at once on the device in 64 bits, and which rows' choice does not hang
    on less than 2^-46 of values of a size of 1, or 2^-46 of them: scores here and in the
    kernel's 64-bit pass are right to some 2^-51."""
    T, E = x.shape
    wide = x.double()
    c = (torch.sigmoid(wide) if scores == "sigmoid" else torch.softmax(wide, 1)) + bias.double()
    held = torch.ones(T, dtype=torch.bool, device=x.device)

    def apart(high, low):  # or one of them is not there
        return (high - low > 2.0**-46 * high.abs().clamp(min=1.0)) | (low == -torch.inf)
    if best < groups:
        top = torch.sort(c.view(T, groups, E // groups), dim=2, descending=True).values[:, :, :2]
        two = torch.where(top > -torch.inf, top, 0.0)
        value = torch.where(top[:, :, 0] > -torch.inf, two.sum(2), -torch.inf)
        order = torch.sort(value, dim=1, descending=True, stable=True)
        size = two.abs().sum(2).gather(1, order.indices[:, best - 1:best + 1]).amax(1).clamp(min=1.0)
        held &= (order.values[:, best - 1] - order.values[:, best] > 2.0**-46 * size) | (order.values[:, best] == -torch.inf)
        chosen = torch.zeros(T, groups, dtype=torch.bool, device=x.device).scatter_(1, order.indices[:, :best], True)
        c = torch.where(chosen.repeat_interleave(E // groups, 1), c, -torch.inf)
    order = torch.sort(c, dim=1, descending=True, stable=True)
    at, v = order.indices[:, :k + 1], order.values[:, :k + 1]
    by_x, by_b = x.gather(1, at), bias[at]
    same = (by_x[:, 1:] == by_x[:, :-1]) & (by_b[:, 1:] == by_b[:, :-1])
    held &= (same | apart(v[:, :-1], v[:, 1:])).all(1)
    return torch.where(order.values[:, :k] > -torch.inf, order.indices[:, :k], -1).int(), held


@pytest.mark.parametrize("seed", range(8))
def test_random_routers(seed):
    """Logits at any place and of any spread, equal, near, and with biases that take scores
    back; biases of any size, and some that leave an expert out or take it always."""
    import random
    rng, g = random.Random(seed), torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    for _ in range(150):
        groups, size = rng.choice([1, 1, 2, 3, 5, 8, 8, 16, 17, 32]), rng.choice([1, 2, 3, 7, 8, 16, 31, 32, 50, 64, 128])
        E, T, scores = groups * size, rng.choice([1, 64, 300]), rng.choice(["sigmoid", "softmax"])
        if E > 1024:
            continue
        best = rng.randint(1, groups)
        k = min(rng.choice([1, 2, 6, 8, 8, 16, 24, 32]), best * size)
        x = normal(T, E) * rng.choice([0.01, 0.5, 1.5, 4, 10]) + rng.choice([0, 0, -5, -9, -14, -20, -30, 12, 20])
        bias = normal(E) * rng.choice([0, 0.001, 0.02, 0.1, 1, 50, 1e4, 1e8])
        kind = rng.choice(["any", "few", "near", "taken back", "taken back", "bf16"])
        if kind == "few":
            x = torch.round(2 * x) / 2
        elif kind == "bf16":
            x = x.bfloat16()
        elif kind != "any":
            x = x[:1] + torch.randint(-30, 31, (T, E), generator=g, device="cuda") * 2.0**-rng.choice([14, 18, 20, 22])
        if kind == "taken back":
            s = torch.sigmoid(x[0].double()) if scores == "sigmoid" else torch.softmax(x[0].double(), 0)
            bias = (rng.choice([0.0, 0.01, 0.5, -1, 3]) - s).float()
        for value in (-1e9, 1e9, LOWEST, -torch.inf):
            if rng.random() < 0.12:
                bias[rng.randrange(E)] = value
        want, held = choose_all(x.float(), bias, k, groups, best, scores)
        got = mxq.moe_route_groups(x, k, bias=bias, scores=scores, groups=groups, best_groups=best).ids
        wrong = (got != want).any(1) & held
        assert not wrong.any(), (kind, E, groups, best, k, scores, int(wrong.sum()), got[wrong][0].tolist(), want[wrong][0].tolist())
