"""The training-step example: it learns, and its gradients are those of the layer.

Gradients are compared with 64-bit autograd through the same layer, with the choice
of experts held fixed.  E4M3 rounds by at most 2^-4, 2^-4/sqrt(3) = 3.6% in the
norm, so a product of two casts is off by at most 7.2% of operands that do not
cancel; the experts' gradients are one such product (and bf16's 0.2%, twice), the
table's and the router's go through two: 8% and 15%.
"""
import importlib.util
from pathlib import Path

import pytest
import torch

import mx_block_quantization_gb300 as mxq
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu
PATH = Path(__file__).resolve().parent.parent / "examples" / "moe_training_step.py"


@pytest.fixture(scope="module")
def example():
    require_gpu()
    spec = importlib.util.spec_from_file_location("moe_training_step", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    yield module
    assert mxq.device_status(clear=True) == 0


def test_learns(example):
    history = example.train(12)
    assert history[-1][0] < 0.8 * history[0][0]
    assert all(b < 1.5 for _, b in history)        # 1 is perfect balance


def test_gradients(example):
    layer = example.MoeLayer(60, 128, 5, 2, seed=3)
    g = torch.Generator().manual_seed(4)
    ids = torch.randint(0, 60, (500,), generator=g).cuda()
    dy = torch.randn(500, 128, generator=g).to(torch.bfloat16).cuda()
    y, balance = layer.forward(ids)
    got = layer.backward(dy, torch.tensor(2.0, device="cuda"))

    table, router, experts = (t.double().cpu().requires_grad_() for t in (layer.table, layer.router, layer.experts))
    x = table[ids.cpu()]
    p = (x @ router.t()).softmax(-1)
    chosen = layer.routing.ids.cpu().long()
    w = p.gather(1, chosen)
    w = w / w.sum(1, keepdim=True)
    out = (torch.einsum("td,tkod->tko", x, experts[chosen]) * w[..., None]).sum(1)
    counts = torch.bincount(chosen.view(-1), minlength=5)
    loss = 5 / (2 * 500**2) * (counts * p.sum(0)).sum()
    ((out * dy.double().cpu()).sum() + 2.0 * loss).backward()

    def off(a, b):
        return float((a.double().cpu() - b).norm() / b.norm())
    assert float(balance) == pytest.approx(float(loss.detach()), rel=1e-5)
    assert off(y, out.detach()) < 0.08
    for a, b, bound in zip(got, (table, router, experts), (0.15, 0.15, 0.08)):
        assert off(a, b.grad) < bound
