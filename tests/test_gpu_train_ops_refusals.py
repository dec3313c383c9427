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


def test_rows_at_no_fixed_distance_and_rows_of_nothing():
    table = torch.randn(10, 8, device="cuda")
    ids = torch.randint(0, 10, (3, 5), device="cuda")
    dy = torch.randn(5, 3, 8, device="cuda").transpose(0, 1)
    for call in (lambda: mxq.embedding(ids, table, out=torch.empty_like(dy)),
                 lambda: mxq.embedding(ids, table, out=torch.empty(5, 3, 8, device="cuda").transpose(0, 1)),
                 lambda: mxq.embedding_backward(ids, dy, 10)):
        with pytest.raises(ValueError, match="rows"):
            call()
    for n, rows in ((5, 0), (0, 8)):
        none = torch.empty(3, n, rows, device="cuda")
        some = ids[:, :n].contiguous()
        assert mxq.embedding(some, table[:, :rows], out=none) is none
        grad = mxq.embedding_backward(some, none, 10)
        assert grad.shape == (10, rows) and (grad == 0).all()
    # single rows and single tokens of wider tensors
    one = torch.randn(1, 1, 20, device="cuda")[..., 3:11]
    got = mxq.embedding_backward(ids[:1, :1].contiguous(), one, 10)
    want = torch.zeros(10, 8, device="cuda")
    want[ids[0, 0]] = one[0, 0]
    assert torch.equal(got, want)


def test_rows_of_a_plan_and_of_its_out_have_to_agree():
    """`rows` beside an `out` of another size was left out of account."""
    ids = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    out = mxq.moe_plan(ids, 2)
    M = out.source.numel()
    with pytest.raises(ValueError, match=str(M + 128)):
        mxq.moe_plan(ids, 2, rows=M + 128, out=out)
    assert mxq.moe_plan(ids, 2, rows=M, out=out) is out
