"""adamw_step as a call: lists that take several launches, and what autograd is told."""
import pytest
import torch

import mx_block_quantization_gb300 as mxq
from tests.gpu_util import require_gpu
from tests.test_gpu_adamw import BF16, HOW, tensors

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    yield
    torch.cuda.empty_cache()
    assert mxq.device_status(clear=True) == 0


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("fault", ["params in params", "params in grads", "copies in params", "one launch", "a copy in moments"])
def test_a_long_list_is_refused_before_anything_moves(fault, bits):
    """Overlaps between tensors of two launches, and within the second one."""
    count = 700
    sizes = [64 + i % 50 for i in range(count)]
    params, grads, copies = tensors(sizes), tensors(sizes, seed=1), [None] * count
    moments = mxq.adamw_moments(params, bits)
    room = torch.randn(500, device="cuda")
    if fault == "params in params":
        params[3], params[600] = room[:sizes[3]], room[8:8 + sizes[600]]
    elif fault == "params in grads":
        params[600], grads[3] = room[:sizes[600]], room[8:8 + sizes[3]]
    elif fault == "copies in params":
        params[3], copies[600] = room[:sizes[3]], room[4:204].view(BF16)[:sizes[600]]
    elif fault == "one launch":
        params[600], params[601] = room[:sizes[600]], room[8:8 + sizes[601]]
    else:  # of a tensor of the first launch
        copies[600] = moments.m.view(BF16)[:sizes[600]]
    before = [p.clone() for p in params], [c if c is None else c.clone() for c in moments]
    with pytest.raises(mxq.MxqError) as e:
        mxq.adamw_step(params, grads, moments, 1, copies=copies, **HOW)
    assert e.value.code == mxq.EOVERLAP
    assert all(torch.equal(a, b) for a, b in zip(params, before[0]))
    assert all(b is None or torch.equal(a, b) for a, b in zip(moments, before[1]))


@pytest.mark.parametrize("bits", [32, 8])
def test_a_graph_that_saved_a_parameter_is_told(bits):
    """As after torch's own optimisers: a backward pass through values that the step has
    changed is an error, not a gradient of the new ones."""
    params = [t.requires_grad_() for t in tensors([100, 300, 200])]
    copies = [p.detach().to(BF16) for p in params[:2]] + [None]
    scale = torch.ones(300, device="cuda", requires_grad=True)
    saved = (params[0] ** 2).sum(), (copies[1] * scale).sum(), (params[2] ** 2).sum()
    moments = mxq.adamw_moments(params, bits)
    grads = tensors([100, 300, 200], seed=1)
    grads[2] = None
    mxq.adamw_step(params, grads, moments, 1, copies=copies, **HOW)
    for y in saved[:2]:
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.backward()
    saved[2].backward()                 # no gradient: left as it is
    assert torch.equal(params[2].grad, 2 * params[2].detach())
    with torch.inference_mode():        # these have no versions
        mxq.adamw_step([params[0] * 1.0], grads[:1], mxq.adamw_moments(params[:1], bits), 1, **HOW)
