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
