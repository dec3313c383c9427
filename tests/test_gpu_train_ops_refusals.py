"""Refusals and shapes of the training operators' Python calls, beside those in the
operators' own files."""
import pytest
import torch

import mx_block_quantization_gb300 as mxq
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    yield
    assert mxq.device_status(clear=True) == 0


def test_counts_past_32_bits_are_refused():
    """ctypes cuts an integer to its lowest bits: these ran as 5 steps, 2 experts, ..."""
    far = 1 << 32
    g, ids = torch.randn(8, 9, device="cuda"), torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    room = mxq.moe_plan(ids, 2)
    for call in (lambda: mxq.orthogonalize(g, steps=far + 5), lambda: mxq.moe_route(g, far + 2),
                 lambda: mxq.moe_plan(ids, far + 2, out=room), lambda: mxq.moe_plan(ids, 2, rows=far + 256),
                 lambda: mxq.embedding_backward(ids[:, 0].contiguous(), g[:4], far + 3, out=torch.empty(3, 9, device="cuda"))):
        with pytest.raises(mxq.MxqError) as e:
            call()
        assert e.value.code == mxq.EBADSHAPE
    with pytest.raises(TypeError):
        mxq.orthogonalize(g, steps=5.0)
