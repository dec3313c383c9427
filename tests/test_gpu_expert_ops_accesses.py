"""Which accesses of the experts' products, grouped routing and AdamW the checked library
tests, as in test_gpu_checked_accesses.py: the first and last element of every buffer that
is not loaded by tensor copies, and the bytes around it."""
import pytest
import torch

import mx_block_quantization_gb300 as mxq
from tests.gpu_util import require_gpu
from tests.test_gpu_checked_accesses import BF16, F32, Workspace, check, room
from tests.test_gpu_moe_linear import ends_of, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    if not mxq.debug_bounds():
        pytest.skip("the checked library's (the suite runs on it as well)")
    yield
    mxq.selftest_watch(0)
    mxq.device_status(clear=True)


def operands(blocks, tail, N, K):
    M, offs = 128 * (sum(blocks) + tail), ends_of(blocks).cuda()
    x = mxq.quantize_2d_dual(normal((M, K), 1, dtype=BF16), offs)
    w = mxq.quantize_2d_dual(normal((len(blocks) * N, K), 2, dtype=BF16))
    return M, room((len(blocks),), torch.int32, fill=offs), x, w


@pytest.mark.parametrize("kind", [F32, BF16])
@pytest.mark.parametrize("blocks,tail,N,K,pad", [([1, 2], 0, 128, 128, 0), ([3, 0, 5], 0, 384, 256, 3), ([1, 4], 2, 256, 128, 1)])
def test_linear(blocks, tail, N, K, pad, kind):
    M, offs, x, w = operands(blocks, tail, N, K)
    y, z, residual, bias = room((M, N), kind, pad), room((M, N), kind, pad + 1), room((M, N), kind, pad), room((len(blocks), N))
    call = lambda: mxq.moe_linear(x.q_row, x.s_row, w.q_row.view(-1, N, K), w.s_row, offs, bias=bias, activation="silu",  # noqa: E731
                                  residual=residual, preactivation=True, out=(y, z))
    # rows behind the last group have no residual
    check(call, dict(y=y, z=z, bias=bias, offs=offs, **({} if tail else dict(residual=residual))))


@pytest.mark.parametrize("kind", [F32, BF16])
@pytest.mark.parametrize("accumulate", [False, True])
def test_weight_gradient(kind, accumulate):
    M, offs, x, _ = operands([2, 0, 3], 1, 128, 256)
    dz = mxq.quantize_2d_dual(normal((M, 384), 3, dtype=BF16), offs)
    # an empty group's matrix is not touched when it is added to: the last one is not empty
    dw = room((3, 384, 256), kind, 5)
    check(lambda: mxq.moe_weight_gradient(dz.q_col, dz.s_col, x.q_col, x.s_col, offs, out=dw, accumulate=accumulate), dict(dw=dw, offs=offs))


@pytest.mark.parametrize("kind", [F32, BF16])
@pytest.mark.parametrize("blocks,N,pad", [([1], 128, 0), ([3, 0, 2], 384, 0), ([2, 1], 256, 3)])
def test_epilogue_gradient(monkeypatch, blocks, N, pad, kind):
    ws = Workspace(monkeypatch)
    M, offs = 128 * sum(blocks), room((len(blocks),), torch.int32, fill=ends_of(blocks).cuda())
    dy, z, dz, db = room((M, N), kind, pad), room((M, N), kind, pad), room((M, N), kind, pad), room((len(blocks), N))
    check(lambda: mxq.moe_linear_backward(dy, z, offs, activation="gelu", out=(dz, db)), dict(dy=dy, z=z, dz=dz, dbias=db, offs=offs), ws,
          [("sums", 0), ("sums", M // 128 * N * 4 - 4)])


@pytest.mark.parametrize("kind", [F32, BF16])
@pytest.mark.parametrize("scores", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,k,groups,best,pad", [(300, 8, 2, 2, 1, 1), (20, 30, 3, 5, 2, 0), (200, 40, 4, 1, 1, 3), (77, 256, 8, 8, 4, 0), (40, 600, 5, 30, 9, 0)])
def test_routing(monkeypatch, T, E, k, groups, best, pad, scores, kind):
    ws = Workspace(monkeypatch)
    x, bias = room((T, E), kind, pad, torch.randn(T, E, device="cuda")), room((E,))
    mask = room((T,), torch.uint8, fill=torch.ones(T))
    out = mxq.Routing(room((T, k)), room((T, k), torch.int32), room((E,), torch.int32), torch.zeros((), device="cuda"),
                      torch.zeros((), dtype=torch.int32, device="cuda"))
    at_once = 32 if E <= 256 else 16 if E <= 512 else 8
    blocks = -(-T // at_once)
    parts = []
    if blocks > 1:
        c, n, loss = 4 * blocks * E, 8 * blocks * E, 8 * blocks * E + 4 * blocks + 4
        parts = [("p", 0), ("p", c - 4), ("c", c), ("c", n - 4), ("n", n), ("n", n + 4 * blocks - 4), ("loss", loss),
                 ("loss", loss + 4 * (-(-E // 32) - 1))]
    how = dict(bias=bias, scores=scores, groups=groups, best_groups=best, mask=mask)
    check(lambda: mxq.moe_route_groups(x, k, out=out, **how),
          dict(logits=x, mask=mask, bias=bias, weights=out.weights, ids=out.ids, counts=out.counts), ws, parts)
    mxq.moe_route_groups(x, k, out=out, **how)
    dw, dl = room((T, k), fill=torch.randn(T, k, device="cuda")), torch.ones((), device="cuda")
    dx = room((T, E), kind, pad)
    check(lambda: mxq.moe_route_groups_backward(x, out, dw, dl, mask=mask, scores=scores, out=dx),
          dict(logits=x, mask=mask, ids=out.ids, counts=out.counts, dweights=dw, dlogits=dx))


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("kind,gkind", [(F32, BF16), (BF16, F32)])
@pytest.mark.parametrize("sizes,at", [((5000, 4096), 0), ((5000, 2049), 1), ((31, 130), 0)])
def test_adamw(sizes, at, kind, gkind, bits):
    one = lambda n, dtype: room((n + at,), dtype)[at:]  # noqa: E731
    params, grads, copies = ([one(n, d) for n in sizes] for d in (kind, gkind, BF16))
    total = sum(-(-n // 128) * 128 for n in sizes)
    whole = torch.uint8 if bits == 8 else F32
    moments = mxq.Moments(room((total,), whole), room((total,), whole), *((room((total // 32,), torch.uint8), room((total // 32,), torch.uint8))
                                                                         if bits == 8 else (None, None)))
    named = {f"{n}{i}": t for n, ts in (("p", params), ("g", grads), ("c", copies)) for i, t in enumerate(ts)}
    # of the moments what belongs to elements: the last tensor's padding is not touched
    used = total - -(-sizes[-1] // 128) * 128 + (-(-sizes[-1] // 32) * 32 if bits == 8 else sizes[-1])
    named.update(m=moments.m[:used], v=moments.v[:used])
    if bits == 8:
        named.update(ms=moments.m_scale[:used // 32], vs=moments.v_scale[:used // 32])
    call = lambda: mxq.adamw_step(params, grads, moments, 1, lr=1e-3, copies=copies)  # noqa: E731
    check(call, named)
