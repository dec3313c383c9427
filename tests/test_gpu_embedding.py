"""embedding and embedding_backward against their definition in 64 bits.

A lookup is one product, rounded once (twice to bf16: in fp32 and then to bf16).
A gradient row of n tokens is a sum in fp32 times the scale: (n + 2) units of
2^-24 of the sum of magnitudes, plus half a unit of bf16 where it is rounded to
it.
"""
import numpy as np
import pytest
import torch

import mx_block_quantization_gb300 as mxq
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    yield
    assert mxq.device_status(clear=True) == 0


def matrix(rows, D, kind, pad=0, seed=0):
    g = torch.Generator().manual_seed(seed + rows * 7 + D)
    return torch.randn(rows, D + pad, generator=g).to(TYPES[kind]).cuda()[:, :D]


def some_ids(T, V, ints, seed=0, skew=True):
    g = np.random.Generator(np.random.PCG64(seed + T + V))
    ids = (V ** g.random(T)).astype(np.int64) - 1 if skew else g.integers(0, V, T)
    return torch.from_numpy((ids * 31 + 5) % V).to(ints).cuda()


@pytest.mark.parametrize("kind,out", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("T,V,D,pad,ints", [
    (1, 1, 1, 0, torch.int64), (8, 100, 64, 0, torch.int64), (5, 7, 33, 2, torch.int32), (300, 50, 1001, 0, torch.int64),
    (17, 1000, 4096, 0, torch.int32), (64, 9, 130, 6, torch.int32), (1000, 333, 24, 0, torch.int64),
])
def test_lookup(T, V, D, pad, ints, kind, out):
    ids, table = some_ids(T, V, ints), matrix(V, D, kind, pad)
    got = mxq.embedding(ids, table, scale=1.7, dtype=TYPES[out])
    want = (table[ids.long()].float() * torch.tensor(1.7, dtype=torch.float32, device="cuda")).to(TYPES[out])
    assert torch.equal(got, want)
    assert torch.equal(mxq.embedding(ids, table), table[ids.long()])


def test_lookup_keeps_the_shape_of_the_ids_and_zeroes_rows_out_of_range():
    table = matrix(20, 40, "bf16")
    ids = some_ids(24, 20, torch.int64).view(2, 3, 4)
    y = mxq.embedding(ids, table)
    assert y.shape == (2, 3, 4, 40) and torch.equal(y, table[ids])
    ids[0, 1, 2], ids[1, 0, 0], ids[1, 2, 3] = 20, -1, 2**40
    z = mxq.embedding(ids, table)
    assert mxq.device_status(clear=True) == mxq.DEV_BADINDEX
    ok = (ids >= 0) & (ids < 20)
    assert torch.equal(z[ok], table[ids[ok]]) and (z[~ok] == 0).all()
    assert mxq.embedding(ids[:0], table).shape == (0, 3, 4, 40)
    out = torch.full((24, 47), 2.0, dtype=torch.bfloat16, device="cuda")
    flat = ids.clamp(0, 19).view(-1)
    mxq.embedding(flat, table, out=out[:, :40])
    assert torch.equal(out[:, :40], table[flat]) and (out[:, 40:] == 2).all()


def check_gradient(ids, dy, V, scale=1.0, padding=None, out=None):
    got = mxq.embedding_backward(ids, dy, V, scale=scale, padding_idx=padding, dtype=out)
    assert got.shape == (V, dy.shape[-1]) and got.dtype == (out or dy.dtype)
    i, g = ids.cpu().numpy().reshape(-1).astype(np.int64), dy.double().cpu().numpy().reshape(ids.numel(), -1)
    keep = (i >= 0) & (i < V) & (i != (-1 if padding is None else padding))
    want, size, n = np.zeros((V, g.shape[1])), np.zeros((V, g.shape[1])), np.zeros((V, 1))
    np.add.at(want, i[keep], scale * g[keep])
    np.add.at(size, i[keep], np.abs(scale * g[keep]))
    np.add.at(n, i[keep], 1)
    half_unit = 2.0**-8 * np.abs(want) if got.dtype == torch.bfloat16 else 0.0
    assert (np.abs(got.double().cpu().numpy() - want) <= (n + 2) * 2.0**-24 * size + half_unit).all()
    assert (got.cpu()[torch.from_numpy(n[:, 0] == 0)] == 0).all()
    return got


@pytest.mark.parametrize("kind,out", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("T,V,D,pad,ints", [
    (1, 1, 1, 0, torch.int64), (1, 5000, 16, 0, torch.int32), (31, 7, 40, 0, torch.int64), (32, 1, 64, 0, torch.int64),
    (33, 1, 65, 3, torch.int32), (64, 2, 8, 0, torch.int64), (100, 1023, 100, 4, torch.int64),
    (1024, 1024, 33, 0, torch.int32), (1025, 1025, 130, 0, torch.int64), (3000, 90, 1001, 3, torch.int32),
    (5000, 70000, 24, 0, torch.int64), (2049, 300, 2048, 0, torch.int32), (777, 31, 4104, 0, torch.int64),
])
def test_gradient(T, V, D, pad, ints, kind, out):
    check_gradient(some_ids(T, V, ints), matrix(T, D, kind, pad), V, scale=2.5, out=TYPES[out])


def test_gradient_with_padding_and_ids_out_of_range():
    ids = some_ids(900, 40, torch.int64)
    check_gradient(ids, matrix(900, 48, "f32"), 40, padding=int(ids[0]))
    bad = ids.clone()
    bad[::7], bad[5], bad[6] = 40, -3, 2**33
    check_gradient(bad, matrix(900, 48, "f32"), 40, padding=3)
    assert mxq.device_status(clear=True) == mxq.DEV_BADINDEX
    every = torch.full((100,), 3, dtype=torch.int32, device="cuda")
    assert (mxq.embedding_backward(every, matrix(100, 8, "bf16"), 5, padding_idx=3) == 0).all()


def test_gradient_many_tokens_uniform_and_one_id():
    check_gradient(some_ids(200003, 3000, torch.int32, skew=False), matrix(200003, 16, "f32"), 3000)
    check_gradient(torch.full((70001,), 11, dtype=torch.int64, device="cuda"), matrix(70001, 40, "f32"), 12)


def test_gradient_of_a_large_vocabulary():
    V = (1 << 20) + 3                               # three digits
    ids = some_ids(4000, V, torch.int64, skew=False)
    ids[:50] = V - 1
    check_gradient(ids, matrix(4000, 8, "f32"), V)


def test_gradient_against_differences():
    """The loss sum(embedding * dy) is linear in the table: its difference along a
    direction is the product with the gradient."""
    ids = some_ids(50, 12, torch.int64).view(5, 10)
    dy = matrix(50, 16, "f32").contiguous().view(5, 10, 16)
    table, way = matrix(12, 16, "f32", seed=1), matrix(12, 16, "f32", seed=2)
    grad = mxq.embedding_backward(ids, dy, 12, scale=0.5)

    def loss(t):
        return (0.5 * t.double()[ids] * dy.double()).sum()
    want = (loss(table.double() + way.double()) - loss(table.double() - way.double())) / 2
    assert float((grad.double() * way.double()).sum()) == pytest.approx(float(want), rel=1e-5, abs=1e-4)


def test_same_bits_and_streams_and_empty():
    ids, dy = some_ids(9000, 700, torch.int64), matrix(9000, 96, "bf16")
    a = mxq.embedding_backward(ids, dy, 700)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = mxq.embedding_backward(ids, dy, 700, stream=side)
    side.synchronize()
    assert torch.equal(a, b) and torch.equal(a, mxq.embedding_backward(ids, dy, 700))
    wide = torch.full((700, 100), 3.0, dtype=torch.bfloat16, device="cuda")
    mxq.embedding_backward(ids, dy, 700, out=wide[:, :96])
    assert torch.equal(wide[:, :96], a) and (wide[:, 96:] == 3).all()
    assert (mxq.embedding_backward(ids[:0], dy[:0], 9) == 0).all()
    assert mxq.embedding_backward(ids[:0], dy[:0], 0).shape == (0, 96)


def test_refusals():
    ids, dy, table = some_ids(10, 6, torch.int64), matrix(10, 8, "f32"), matrix(6, 8, "f32")
    for bad in (ids.cpu(), ids.short(), ids.float()):
        with pytest.raises(ValueError):
            mxq.embedding(bad, table)
    for bad in (table.half(), table.cpu(), table.t()):
        with pytest.raises(ValueError):
            mxq.embedding(ids, bad)
    with pytest.raises(ValueError):
        mxq.embedding(ids, table, dtype=torch.float16)
    with pytest.raises(ValueError):
        mxq.embedding(ids, table, out=torch.empty(9, 8, device="cuda"))
    with pytest.raises(ValueError):
        mxq.embedding_backward(ids, dy[:9], 6)
    for padding in (-1, 6):
        with pytest.raises(ValueError):
            mxq.embedding_backward(ids, dy, 6, padding_idx=padding)
    with pytest.raises((mxq.MxqError, RuntimeError)):
        mxq.embedding_backward(ids, dy, -1)
    with pytest.raises(mxq.MxqError) as e:
        mxq.embedding_backward(ids, dy, 10, out=dy)
    assert e.value.code == mxq.EOVERLAP
