"""What the training operators' Python calls do before they reach the C entries, by
stand-ins, without a GPU."""
from types import SimpleNamespace

import pytest
import torch

from mx_block_quantization_gb300 import training


def test_a_stream_of_another_device_is_refused():
    """It used to be dropped: the call then ran on the tensors' device's current stream."""
    other = SimpleNamespace(device=torch.device("cuda", 1))
    with pytest.raises(ValueError, match="cuda:1"):
        training._elsewhere(torch.device("cuda", 0), other)


def test_a_stream_of_the_tensors_device_is_entered(monkeypatch):
    own = SimpleNamespace(device=torch.device("cuda", 1))
    monkeypatch.setattr(torch.cuda, "stream", lambda s: ("entered", s))
    assert training._elsewhere(torch.device("cuda", 1), own) == ("entered", own)


def test_without_a_stream_the_tensors_device_is_current(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    monkeypatch.setattr(torch.cuda, "device", lambda d: ("device", d))
    assert training._elsewhere(torch.device("cuda", 1), None) is None
    assert training._elsewhere(torch.device("cuda", 0), None) == ("device", torch.device("cuda", 0))


@pytest.mark.parametrize("args", [(10, 2, 1 << 32 | 8), (10, 1 << 32 | 2, 8), (1 << 64 | 10, 2, 8), (10, -(1 << 32) + 2, 8)])
def test_counts_past_32_bits_are_refused(args):
    """ctypes cuts an integer to its lowest bits: these were answered as (10, 2, 8)."""
    import mx_block_quantization_gb300 as mxq
    if not mxq.LIB_PATH.exists():
        import __graft_entry__
        __graft_entry__.build()
    assert mxq.moe_rows(10, 2, 8) == 1024
    with pytest.raises(mxq.MxqError) as e:
        mxq.moe_rows(*args)
    assert e.value.code == mxq.EBADSHAPE


def test_rows_of_a_tensor_share_its_memory_or_are_refused():
    """Rows at no fixed distance were torch's RuntimeError, and rows of no elements too."""
    x = torch.arange(2 * 3 * 8.0).view(2, 3, 8)
    for t in (x, x[..., 1:6], x[:, :1], x[:1], x[0], x[0, 1]):
        D = t.shape[-1]
        r = training._rows_of(t, "x", t.numel() // D, D)
        assert torch.equal(r, t.reshape(-1, D)) and r.data_ptr() == t.data_ptr()
    for t in (x.transpose(0, 1), x[:, :2], x.permute(1, 0, 2)[..., :4]):
        with pytest.raises(ValueError, match="x must have rows"):
            training._rows_of(t, "x", t.shape[0] * t.shape[1], t.shape[2])
    for shape in ((2, 3, 0), (0, 3, 8), (2, 0, 8), (0,), (0, 0)):
        T = 1
        for n in shape[:-1]:
            T *= n
        assert training._rows_of(torch.empty(shape), "x", T, shape[-1]).shape == (T, shape[-1])


def test_a_release_library_takes_a_watched_address_and_does_nothing():
    import mx_block_quantization_gb300 as mxq
    if not mxq.debug_bounds():
        mxq.selftest_watch(1 << 40)
        mxq.selftest_watch()
