"""orthogonalize writes the elements of `out` and nothing else, and reads nothing that it
has not written."""
import pytest
import torch

import mx_block_quantization_gb300 as mxq
from mx_block_quantization_gb300 import training
from tests.gpu_util import require_gpu
from tests.test_gpu_orthogonalize import momentum

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    yield
    assert mxq.device_status(clear=True) == 0


@pytest.mark.parametrize("m,n", [(20, 7), (100, 121), (70, 120), (200, 333), (333, 201), (5, 9), (90, 100), (300, 260), (40, 1001)])
@pytest.mark.parametrize("pitch", [8, 16, 1, 2])     # rows' distance: a multiple of it
@pytest.mark.parametrize("shift", [0, 8, 1])
def test_nothing_beside_the_rows(m, n, pitch, shift):
    """Rows with gaps, in one of their own buffer's ends: the last row ends where the
    memory does that belongs to the result."""
    g = momentum(2, m, n)
    want = mxq.orthogonalize(g)
    ld = -(-(n + 1) // pitch) * pitch
    stride = m * ld + 8
    end = shift + stride + (m - 1) * ld + n
    room = torch.full((end + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = room.as_strided((2, m, n), (stride, ld, 1), shift)
    mxq.orthogonalize(g, out=out)
    assert torch.equal(out, want)
    out.fill_(7.0)
    assert (room == 7).all()


@pytest.mark.parametrize("batch,m,n", [(1, 20, 7), (2, 50, 33), (1, 130, 201), (3, 201, 130), (1, 300, 5001), (1, 5001, 300),
                                       (1, 41, 9001), (1, 70, 71)])
@pytest.mark.parametrize("co", [(3.4445, -4.775, 2.0315), (1.5, -0.5, 0.0)])
def test_workspaces_may_hold_anything(monkeypatch, batch, m, n, co):
    """Bytes of 0xFF are NaN in every type that the workspace holds."""
    g = momentum(batch, m, n)
    want = mxq.orthogonalize(g, coefficients=co)

    def poisoned(size, what, device):
        t = torch.full((size,), 0xFF, dtype=torch.uint8, device=device)
        return t, t.data_ptr()

    monkeypatch.setattr(training, "_workspace", poisoned)
    assert torch.equal(mxq.orthogonalize(g, coefficients=co), want)
