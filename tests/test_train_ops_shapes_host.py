"""Shapes that the training operators' C entries state as allowed, on the host."""
import pytest

import mx_block_quantization_gb300 as mxq


@pytest.fixture(scope="module")
def L():
    if not mxq.LIB_PATH.exists():
        import __graft_entry__
        __graft_entry__.build()
    return mxq.lib()


@pytest.mark.parametrize("batch,m,n", [(64, 1 << 20, 1), (64, 1, 1 << 20), (64, 1 << 20, 16), (200, 600000, 64),
                                       (65535, 1 << 17, 4), (65535, 256, 1 << 20), (65535, 1, 1)])
def test_orthogonalize_takes_stacks_of_very_long_matrices(L, batch, m, n):
    """No product has the longer side squared."""
    assert L.mxq_orthogonalize_workspace(batch, m, n) >= 4 * batch * m * n  # X twice, in fp16


@pytest.mark.parametrize("batch,m,n", [(65535, 1 << 20, 1 << 20), (65535, 1 << 20, 1 << 15), (4096, 1 << 17, 1 << 18)])
def test_orthogonalize_refuses_more_tiles_than_it_counts(L, batch, m, n):
    assert L.mxq_orthogonalize_workspace(batch, m, n) == mxq.EBADSHAPE
