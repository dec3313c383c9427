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
