"""moe_route_groups takes about as long whatever single biases are and however small the
scores: a near tie is done again in 64 bits, and what makes every row look like one costs
ten times the time of the call.  Times are compared with the same batch's of usual values
in the same test, the shortest of several each; the margin is a factor of two.
"""
import math

import pytest
import torch

import mx_block_quantization_gb300 as mxq
from tests.gpu_util import require_gpu
from tests.test_gpu_moe_route_groups import Case

pytestmark = pytest.mark.gpu
T, E = 131072, 256


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    yield
    torch.cuda.empty_cache()
    assert mxq.device_status(clear=True) == 0


def shortest(call):
    """Microseconds of a call among eight of them, the best of six times."""
    best = math.inf
    for i in range(7):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(8):
            call()
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b) * 125 if i else math.inf)
    return best


def times(x, k, biases, **how):
    return [shortest(lambda: mxq.moe_route_groups(x, k, bias=b, **how)) for b in biases]


@pytest.mark.parametrize("scores", ["sigmoid", "softmax"])
@pytest.mark.parametrize("e,groups,best", [(E, 8, 4), (E, 1, 1), (512, 8, 4)])
def test_a_bias_that_leaves_an_expert_out_or_takes_it_always(e, groups, best, scores):
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(T, e, generator=g, device="cuda") * 1.5
    usual = torch.randn(e, generator=g, device="cuda") * 0.02
    biases = [usual]
    for value in (-math.inf, -1e9, torch.finfo(torch.float32).min, 1e9, math.inf, math.nan):
        b = usual.clone()
        b[77] = value
        biases.append(b)
    took = times(x, 8, biases, scores=scores, groups=groups, best_groups=best)
    assert max(took) < 2 * took[0], took
    for b in biases[1:]:
        Case(300, e, 8, groups, best, scores, x=x[:300].cpu(), bias=b.cpu()).check(exact=False)


@pytest.mark.parametrize("bias", [None, 0.0, -0.01])
@pytest.mark.parametrize("e,groups,best", [(E, 8, 4), (E, 1, 1), (512, 8, 4)])
def test_small_scores(e, groups, best, bias):
    """Sigmoid scores of 1e-6, and of 1e-9, are as far apart for their size as usual ones.  A
    bias of all experts leaves them what fp32 has behind its size: with 0.01 1e-9 of them, so
    that there only the larger ones are compared."""
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(T, e, generator=g, device="cuda") * 1.5
    bias = None if bias is None else torch.full((e,), bias, device="cuda")
    shifts = [0.0, -14.0, -20.0] if bias is None or not bias.any() else [0.0, -10.0]
    took = [times(x + y, 8, [bias], scores="sigmoid", groups=groups, best_groups=best)[0] for y in shifts]
    assert max(took) < 2 * took[0], took
    for y in shifts[1:]:
        Case(300, e, 8, groups, best, "sigmoid", x=x[:300].cpu() + y, bias=None if bias is None else bias.cpu()).check(exact=False)


@pytest.mark.parametrize("scores", ["sigmoid", "softmax"])
@pytest.mark.parametrize("e,groups,best", [(250, 5, 3), (512, 1, 1), (512, 8, 4), (1000, 1, 1)])
def test_the_most_choices(e, groups, best, scores):
    """32 experts a token take four times as many rounds as 8, and the search for the 32nd."""
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(T, e, generator=g, device="cuda") * 1.5
    bias = torch.randn(e, generator=g, device="cuda") * 0.02
    how = dict(scores=scores, groups=groups, best_groups=best)
    took = [times(x, k, [bias], **how)[0] for k in (8, 20, 32)]
    assert max(took) < 4 * took[0], took
    for k in (20, 32):
        Case(300, e, k, groups, best, scores, x=x[:300].cpu(), bias=bias.cpu()).check(exact=False)
