"""moe_linear_backward without an activation: dz in a buffer of its own."""
import pytest
import torch

import mx_block_quantization_gb300 as mxq
from tests.gpu_util import require_gpu
from tests.test_gpu_moe_linear import BF16, F32, ends_of, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    yield
    torch.cuda.empty_cache()
    assert mxq.device_status(clear=True) == 0


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("blocks,tail,N", [([1], 0, 128), ([3, 0, 2], 2, 384), ([0], 1, 128)])
def test_rows_behind_the_last_group_without_an_activation(blocks, tail, N, dtype):
    """dz is dy: where it is dy itself its last rows stay as they are, in a buffer of its own
    they are 0 as with an activation.  Their values are in no sum.  dbias is a sum of at most
    128 b terms d of fp32; at another pitch they are added in another order, so that two of
    them are at most 2 (128 b) 2^-24 of the sum of |d| apart."""
    M, offs, end = 128 * (sum(blocks) + tail), ends_of(blocks).cuda(), 128 * sum(blocks)
    dy = normal((M, N), 1, dtype=dtype)
    kept = dy.clone()
    got, dbias = mxq.moe_linear_backward(dy, offs=offs)
    assert got is dy and torch.equal(dy, kept)
    got, again = mxq.moe_linear_backward(dy, offs=offs, out=(dy, torch.empty_like(dbias)))
    assert got is dy and torch.equal(dy, kept) and torch.equal(again, dbias)
    room = torch.full((M, N + 5), 3.0, dtype=dtype, device="cuda")
    dz, own = mxq.moe_linear_backward(dy, offs=offs, out=(room[:, 2:N + 2], torch.empty_like(dbias)))
    assert torch.equal(dz[:end], dy[:end]) and not dz[end:].any()
    lo = 0
    for e, b in enumerate(blocks):
        hi = lo + 128 * b
        assert bool(((own[e] - dbias[e]).double().abs() <= 2 * 128 * b * 2.0**-24 * dy[lo:hi].double().abs().sum(0)).all())
        lo = hi
    assert bool((room[:, :2] == 3).all()) and bool((room[:, N + 2:] == 3).all()) and torch.equal(dy, kept)
    with pytest.raises(mxq.MxqError) as e:
        mxq.moe_linear_backward(room[:, :N], offs=offs, out=(room[:, 2:N + 2], torch.empty_like(dbias)))
    assert e.value.code == mxq.EOVERLAP


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("activation", [None, "relu", "silu", "gelu"])
@pytest.mark.parametrize("pad", [0, 1, 8])
def test_in_place_of_dy(activation, dtype, pad):
    """dz over dy, with many blocks of the grid side by side in a row: the bits of a call
    with buffers of their own at the same pitch."""
    blocks, N = [9, 0, 30, 1], 1152
    M, offs = 128 * (sum(blocks) + 3), ends_of(blocks).cuda()
    both = torch.empty(2, M, N + pad, dtype=dtype, device="cuda")
    both[0, :, :N] = normal((M, N), 1, dtype=dtype)
    both[1, :, :N] = normal((M, N), 2, 2.0, dtype=dtype)
    dy, z = both[0, :, :N], both[1, :, :N]
    out = torch.empty_like(both[0])[:, :N], torch.empty(4, N, device="cuda")
    dz, dbias = mxq.moe_linear_backward(dy, z, offs, activation=activation, out=out)
    over = dy[:]  # another tensor of the same memory
    for _ in range(2 if activation is None else 1):  # without an activation again and again
        got, again = mxq.moe_linear_backward(dy, z, offs, activation=activation, out=(over, torch.empty_like(dbias)))
        assert torch.equal(got, dz) and torch.equal(again, dbias)
