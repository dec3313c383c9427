"""The experts' products, grouped routing and AdamW where offsets pass 32 bits: what lies
behind 2^31 elements comes out as in a call of its own."""
import pytest
import torch

import mx_block_quantization_gb300 as mxq
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()
    yield
    torch.cuda.empty_cache()
    assert mxq.device_status(clear=True) == 0


def normal(shape, seed, dtype=BF16):
    return torch.randn(shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda").to(dtype)


def test_rows_of_a_product():
    M, N, K = 1048576 + 256, 2176, 128
    assert M * N > 2**31
    w = mxq.quantize_2d_dual(normal((3 * N, K), 1))
    x = torch.zeros(M, K, dtype=BF16, device="cuda")
    x[-512:], x[:256] = normal((512, K), 2), normal((256, K), 3)
    offs = torch.tensor([256, M - 256, M], dtype=torch.int32, device="cuda")
    c, bias = mxq.quantize_2d_dual(x, offs), normal((3, N), 4, torch.float32)
    y, z = mxq.moe_linear(c.q_row, c.s_row, w.q_row.view(3, N, K), w.s_row, offs, bias=bias, activation="silu", preactivation=True)
    for lo, hi, e in ((0, 256, 0), (M - 512, M - 256, 1), (M - 256, M, 2)):
        part = mxq.quantize_2d_dual(x[lo:hi].contiguous())
        want = mxq.moe_linear(part.q_row, part.s_row, w.q_row[e * N:(e + 1) * N], w.s_row.view(3, -1)[e].contiguous(), bias=bias[e],
                              activation="silu", preactivation=True)
        assert torch.equal(y[lo:hi], want[0]) and torch.equal(z[lo:hi], want[1])
    dz, dbias = mxq.moe_linear_backward(y, z, offs, activation="silu")
    want, wbias = mxq.moe_linear_backward(y[-256:], z[-256:], activation="silu")
    assert torch.equal(dz[-256:], want) and torch.equal(dbias[2], wbias)


def test_matrices_of_a_weight_gradient():
    G, N = 1024, 1536
    assert G * N * N > 2**31
    offs = torch.full((G,), 128, dtype=torch.int32, device="cuda")
    offs[-1] = 384
    a, b = (mxq.quantize_2d_dual(normal((384, N), s), offs) for s in (5, 6))
    dw = mxq.moe_weight_gradient(a.q_col, a.s_col, b.q_col, b.s_col, offs)
    a, b = (mxq.quantize_2d_dual(normal((384, N), s)[128:].contiguous()) for s in (5, 6))
    assert torch.equal(dw[-1], mxq.moe_weight_gradient(a.q_col, a.s_col, b.q_col, b.s_col))
    assert not dw[1:-1].any() and dw[0].any()


@pytest.mark.parametrize("scores", ["sigmoid", "softmax"])
def test_tokens_of_a_router(scores):
    T, E, k = 2**23 + 77, 256, 4
    logits = torch.zeros(T, E, dtype=BF16, device="cuda")
    logits[-77:] = normal((77, E), 7)
    how = dict(bias=normal((E,), 8, torch.float32), scores=scores, groups=8, best_groups=3)
    mask = torch.zeros(T, dtype=torch.bool, device="cuda")
    mask[-77:] = True
    r, part = mxq.moe_route_groups(logits, k, mask=mask, **how), mxq.moe_route_groups(logits[-77:], k, **how)
    assert torch.equal(r.ids[-77:], part.ids) and torch.equal(r.weights[-77:], part.weights) and torch.equal(r.counts, part.counts)
    assert bool((r.ids[:-77] == -1).all())
    dw = normal((T, k), 9, torch.float32)
    got = mxq.moe_route_groups_backward(logits, r, dw, mask=mask, scores=scores)
    want = mxq.moe_route_groups_backward(logits[-77:], part, dw[-77:].contiguous(), scores=scores)
    assert torch.equal(got[-77:], want) and not got[:-77].any()


@pytest.mark.parametrize("bits", [8, 32])
def test_elements_of_a_tensor(bits):
    n = 2**31 + 4999
    p, g = torch.zeros(n, dtype=BF16, device="cuda"), torch.zeros(n, dtype=BF16, device="cuda")
    p[-4999:], g[-4999:] = normal((4999,), 10), normal((4999,), 11)
    few = [p[-4999:].clone()]
    moments, few_moments = mxq.adamw_moments([p], bits), mxq.adamw_moments(few, bits)
    mxq.adamw_step([p], [g], moments, 1, lr=0.01)
    mxq.adamw_step(few, [g[-4999:].clone()], few_moments, 1, lr=0.01)
    assert torch.equal(p[-4999:], few[0]) and not p[:-4999].any()
    if bits == 32:
        assert torch.equal(moments.m[2**31:2**31 + 4999], few_moments.m[:4999])
    else:  # the random bits are of the place, the scales are not
        assert torch.equal(moments.m_scale[2**26:], few_moments.m_scale) and torch.equal(moments.v_scale[2**26:], few_moments.v_scale)
