"""Edges of the training operators: sizes at the borders of their variants, offsets
past 32 bits, and elements that are not finite.

orthogonalize is held to 4.8e-3 in the relative Frobenius norm (a rounding of the
result to bf16, and 2^-12 / sqrt(3) for each of the four operands of five steps;
a gram matrix in slices of K adds its fp32 sums in another order, 2^-24 of them).
Lookups, dispatched rows and sums of whole numbers are exact.
"""
import numpy as np
import pytest
import torch

import mx_block_quantization_gb300 as mxq
from tests.gpu_util import require_gpu
from tests.test_gpu_moe_exchange import check_plan, routing
from tests.test_gpu_moe_route import check, logits
from tests.test_gpu_orthogonalize import BOUND, iteration, momentum, off

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    yield
    torch.cuda.empty_cache()
    assert mxq.device_status(clear=True) == 0


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("batch,m,n,pad", [
    (1, 64, 8192, 0), (1, 8192, 64, 0), (1, 65, 8192, 3), (1, 300, 5000, 0), (1, 5001, 300, 0), (2, 40, 9000, 0),
    (3, 128, 6000, 8), (1, 520, 12000, 0), (1, 1, 20000, 0),
])
def test_gram_matrices_in_slices(batch, m, n, pad, kind):
    g = momentum(batch, m, n, kind, pad)
    got = mxq.orthogonalize(g)
    assert off(got, iteration(g)) <= BOUND
    assert torch.equal(got, mxq.orthogonalize(g))
    assert torch.equal(got, mxq.orthogonalize(g.contiguous()))


@pytest.mark.parametrize("m,n", [(2, 2), (63, 64), (64, 65), (65, 64), (72, 4104), (130, 40), (256, 264)])
def test_rows_with_and_without_gaps_between_them(m, n):
    """One run of elements, strided rows and strided matrices of the same values."""
    g = momentum(3, m, n)
    want = mxq.orthogonalize(g)
    assert off(want, iteration(g)) <= BOUND
    rows = torch.full((3, m, n + 5), float("nan"), device="cuda")
    rows[..., :n] = g
    stacks = torch.full((3, m + 1, n), float("nan"), device="cuda")
    stacks[:, :m] = g
    for other in (rows[..., :n], stacks[:, :m]):
        # the norm's sum may be in another order
        assert off(mxq.orthogonalize(other), want.double().cpu()) <= 2 * BOUND


def test_matrices_far_apart():
    far = (1 << 31) + 4096                       # elements between the two
    room = torch.empty(far + 200 * 128, dtype=torch.bfloat16, device="cuda")
    g = room.as_strided((2, 200, 128), (far, 128, 1))
    g.copy_(momentum(2, 200, 128, "bf16"))
    want = mxq.orthogonalize(g.contiguous())
    assert torch.equal(mxq.orthogonalize(g), want)
    out = torch.empty_like(room).as_strided((2, 200, 128), (far, 128, 1))
    mxq.orthogonalize(g, out=out)
    assert torch.equal(out, want)


@pytest.mark.parametrize("T", [1023, 1024, 1026, 4095, 4096, 4097, 16383, 16384, 16385, 65537])
@pytest.mark.parametrize("V", [1, 255, 256, 257, 65536, 65537])
def test_table_gradient_at_the_borders_of_the_sort(T, V):
    """Sums of whole numbers below 2^24 are exact in any order."""
    g = torch.Generator().manual_seed(T + V)
    ids = torch.randint(0, V, (T,), generator=g, dtype=torch.int32).cuda()
    dy = torch.randint(-16, 17, (T, 12), generator=g).float().cuda()
    want = torch.zeros(V, 12, dtype=torch.float64).index_add_(0, ids.cpu().long(), dy.cpu().double())
    assert torch.equal(mxq.embedding_backward(ids, dy, V).cpu().double(), want)
    room = torch.full((V, 15), 7.0, device="cuda")
    mxq.embedding_backward(ids.long(), dy, V, out=room[:, :12])
    assert torch.equal(room[:, :12].cpu().double(), want) and (room[:, 12:] == 7).all()


def test_table_past_32_bits():
    V, D = 300_000, 8192                          # 2.46e9 elements
    table = torch.empty(V, D, dtype=torch.bfloat16, device="cuda")
    ids = torch.tensor([V - 1, 0, V - 2, 262_143, 262_144, V - 1], device="cuda")
    table[ids] = torch.randn(6, D, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    assert torch.equal(mxq.embedding(ids, table), table[ids])
    dy = torch.randint(-8, 9, (6, D), generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    table.fill_(3.0)
    mxq.embedding_backward(ids, dy, V, out=table)
    want = torch.zeros(V, dtype=torch.bool, device="cuda").index_fill_(0, ids, True)
    assert torch.equal(table[V - 1], dy[0] + dy[5])
    assert all(torch.equal(table[ids[i]], dy[i]) for i in (1, 2, 3, 4))
    assert int((table != 0).any(1).sum()) == int((want & (table != 0).any(1)).sum()) == 5


def test_expert_rows_past_32_bits():
    T, k, E, D = 40_000, 8, 16, 8192              # 2.6e9 elements of rows
    ids = routing(T, E, k, dropped=0)
    plan = mxq.moe_plan(torch.from_numpy(ids).cuda(), E)
    M = plan.source.numel()
    assert M * D > 1 << 31
    x = torch.randint(-4, 5, (T, D), device="cuda", dtype=torch.int8).to(torch.bfloat16)
    rows = mxq.moe_dispatch(x, plan)
    for r in (0, M // 2, int(plan.offs[-1]) - 129, M - 1):
        i = int(plan.source[r])
        assert torch.equal(rows[r], x[i // k] if i >= 0 else torch.zeros_like(x[0]))
    # k equal rows of each token: the weights' sum times the row, exact in bf16
    w = torch.full((T, k), 0.25, device="cuda")
    assert torch.equal(mxq.moe_combine(rows, plan, w), x * 2)
    dweights = torch.empty(T, k, device="cuda")
    mxq.moe_combine_backward(x, rows, plan, w, out=(torch.empty_like(rows), dweights))
    want = (x.float() ** 2).sum(1, keepdim=True).expand(T, k)
    assert torch.equal(dweights, want)            # whole numbers below 2^24


def test_logits_past_32_bits():
    T, E, ld = 40, 64, (1 << 26) + 8              # the last rows start past 2^31 elements
    room = torch.empty((T - 1) * ld + E, dtype=torch.bfloat16, device="cuda")
    x = room.as_strided((T, E), (ld, 1))
    x.copy_(torch.randn(T, E, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16))
    a, b = mxq.moe_route(x, 4), mxq.moe_route(x.contiguous(), 4)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    dw = torch.randn(T, 4, generator=torch.Generator().manual_seed(4)).cuda()
    dl = torch.tensor(1.0, device="cuda")
    d = mxq.moe_route_backward(x, a, dw, dl, out=torch.empty_like(room).as_strided((T, E), (ld, 1)))
    assert torch.equal(d, mxq.moe_route_backward(x.contiguous(), b, dw, dl))


def test_not_finite_rows_stay_by_themselves():
    """Dispatch copies bits; a sum has NaN where one of its own rows has, and a choice
    of weight 0 is still a product (0 * inf)."""
    T, k, E, D = 30, 3, 5, 40
    plan, slots, source = check_plan(routing(T, E, k, dropped=0), E)
    x = torch.randn(T, D, generator=torch.Generator().manual_seed(5)).cuda()
    x[4, 3], x[5, 0], x[6, 1] = float("nan"), float("inf"), float("-inf")
    rows = mxq.moe_dispatch(x, plan)
    live = torch.from_numpy(source >= 0).cuda()
    tokens = torch.from_numpy(source[source >= 0] // k).cuda()
    assert torch.equal(rows[live].view(torch.int32), x[tokens].view(torch.int32))
    w = torch.full((T, k), 0.5, device="cuda")
    w[5, 1] = 0.0
    y = mxq.moe_combine(rows, plan, w)
    bad = torch.zeros(T, D, dtype=torch.bool, device="cuda")
    bad[4, 3] = bad[5, 0] = True
    assert torch.equal(y.isnan(), bad) and y[6, 1] == float("-inf")
    # the filled-up rows are not read, whatever they hold
    clean = mxq.moe_combine(rows, plan, w)
    rows[~live] = float("nan")
    assert torch.equal(mxq.moe_combine(rows, plan, w).view(torch.int32), clean.view(torch.int32))
    _, dweights = mxq.moe_combine_backward(torch.ones_like(x), rows, plan, w)
    assert torch.equal(dweights.isfinite().all(1).cpu(), torch.tensor([t not in (4, 5, 6) for t in range(T)]))


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
def test_masks_of_the_lowest_value(kind):
    """A finite lowest value is a logit like others: chosen last, weight 0."""
    low = torch.finfo(kind).min
    x = torch.full((3, 70), low, dtype=kind, device="cuda")
    x[0, 5] = x[0, 69] = 1.0
    r = mxq.moe_route(x, 3, renorm=False)
    assert r.ids.tolist() == [[5, 69, 0], [0, 1, 2], [0, 1, 2]] and int(r.routed) == 3
    assert r.weights[0].tolist() == [0.5, 0.5, 0.0]
    np.testing.assert_allclose(r.weights[1:].cpu().numpy(), 1 / 70, rtol=2.0**-20)
    d = mxq.moe_route_backward(x, r, torch.ones(3, 3, device="cuda"), torch.tensor(1.0, device="cuda"), renorm=False)
    assert d.isfinite().all()


@pytest.mark.parametrize("batch,m,n,pad", [
    (1, 5, 9, 0), (3, 64, 40, 0), (1, 64, 8192, 0), (2, 65, 130, 0), (1, 300, 520, 4), (4, 600, 257, 0), (1, 200, 7000, 0),
])
def test_coefficients_without_a_square_to_complete(batch, m, n, pad):
    """c zero, and b much larger than c: the polynomial adds b A from memory."""
    g = momentum(batch, m, n, pad=pad)
    for co in ((1.5, -0.5, 0.0), (1.6, -0.65, 0.05)):
        assert off(mxq.orthogonalize(g, coefficients=co), iteration(g, coefficients=co)) <= BOUND


def test_coefficients_without_a_polynomial():
    """b = c = 0 only scales: five times a."""
    g = momentum(1, 90, 150)[0]
    want = g.double().cpu() / g.double().cpu().norm() * 1.125**5
    assert off(mxq.orthogonalize(g, coefficients=(1.125, 0.0, 0.0), eps=0.0), want) <= BOUND


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,D,E,k", [
    (5, 1, 3, 2), (200, 3, 4, 1), (33, 31, 5, 3), (40, 63, 5, 8), (70, 129, 3, 2), (64, 1023, 6, 8), (20, 4089, 4, 2),
    (9, 8183, 3, 3), (7, 16377, 2, 2), (6, 20001, 3, 1), (30, 2050, 9, 8), (30, 4100, 9, 9), (12, 8202, 4, 8),
])
@pytest.mark.parametrize("shift,pad", [(0, 0), (1, 1), (3, 6)])
def test_dispatched_rows_at_any_address(T, D, E, k, shift, pad, kind):
    """Rows that begin anywhere: equal bits inside, nothing written outside."""
    k = min(k, E)
    plan, _, source = check_plan(routing(T, E, k), E)
    M = source.size
    x = torch.randn(T, D + pad + shift, generator=torch.Generator().manual_seed(D)).to(kind).cuda()[:, shift:shift + D]
    room = torch.full((M * (D + pad) + shift + 8,), 7.0, dtype=kind, device="cuda")
    rows = room[shift:shift + M * (D + pad)].view(M, D + pad)
    mxq.moe_dispatch(x, plan, out=rows[:, :D])
    want = torch.zeros(M, D, dtype=kind, device="cuda")
    live = torch.from_numpy(np.flatnonzero(source >= 0)).cuda()
    want[live] = x[torch.from_numpy(source[source >= 0] // k).cuda()]
    assert torch.equal(rows[:, :D], want)
    assert (rows[:, D:] == 7).all() and (room[:shift] == 7).all() and (room[shift + M * (D + pad):] == 7).all()


@pytest.mark.parametrize("types", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("T,V,D", [
    (300, 40, 33), (300, 40, 1001), (70, 9, 4097), (65, 9, 16411), (1, 5, 127), (70000, 50, 128), (70000, 50, 2), (20001, 50, 520),
    (5000, 20, 2052), (90000, 60, 31),
])
@pytest.mark.parametrize("shift,pad", [(0, 0), (1, 2)])
def test_looked_up_rows_at_any_address(T, V, D, shift, pad, types):
    """Rows that begin anywhere, many tokens and few, ids out of range among them."""
    a, b = ({"f32": torch.float32, "bf16": torch.bfloat16}[t] for t in types)
    g = torch.Generator().manual_seed(T + D)
    table = torch.randn(V, D + shift + pad, generator=g).to(a).cuda()[:, shift:shift + D]
    ids = torch.randint(0, V, (T,), generator=g).cuda()
    room = torch.full((T * (D + pad) + shift + 8,), 7.0, dtype=b, device="cuda")
    rows = room[shift:shift + T * (D + pad)].view(T, D + pad)
    mxq.embedding(ids, table, out=rows[:, :D])
    assert torch.equal(rows[:, :D], table[ids].to(b))
    assert (rows[:, D:] == 7).all() and (room[:shift] == 7).all() and (room[shift + T * (D + pad):] == 7).all()
    ids[T // 2], ids[0] = V, -7
    got = mxq.embedding(ids, table, dtype=b)
    assert mxq.device_status(clear=True) == mxq.DEV_BADINDEX
    want = table[ids.clamp(0, V - 1)].to(b)
    want[T // 2], want[0] = 0, 0
    assert torch.equal(got, want)


@pytest.mark.parametrize("batch,m,n", [(4, 4160, 256), (1, 3316, 196), (2, 70, 8000), (1, 96, 4145)])
def test_long_matrices_are_as_exact_as_square_ones(batch, m, n):
    """Nearly equal singular values: all of a diagonal's elements round the same way.
    What is left of the diagonals is put back, so the four operands' roundings are
    those of a random matrix's off-diagonal elements, 2^-12 / sqrt(3) each, five
    times and without a common sign: 6.3e-4 added in squares, twice that with the
    iteration's slope, beside the 1.7e-3 of bf16: 2.2e-3."""
    g = momentum(batch, m, n)
    assert off(mxq.orthogonalize(g), iteration(g)) <= 2.2e-3


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("T,E,k,pad", [
    (1, 1, 1, 0), (1, 8, 8, 0), (127, 5, 2, 0), (128, 8, 2, 1), (129, 8, 1, 0), (130, 9, 9, 0), (300, 16, 16, 0), (257, 12, 3, 3),
    (5000, 8, 2, 0), (40003, 16, 4, 0), (3, 15, 10, 1), (200, 17, 5, 0), (1000, 32, 32, 0), (131, 31, 9, 1),
])
@pytest.mark.parametrize("renorm", [False, True])
def test_few_experts(T, E, k, pad, kind, renorm):
    x = logits(T, E, kind, pad)
    check(x, k, renorm=renorm)
    mask = torch.rand(T, generator=torch.Generator().manual_seed(T)).cuda() > 0.3
    check(x, k, mask=mask, renorm=renorm)


@pytest.mark.parametrize("E,k", [(7, 3), (8, 8), (16, 5), (30, 12)])
@pytest.mark.parametrize("renorm", [False, True])
def test_few_experts_agree_with_many(E, k, renorm):
    """Experts of -inf added up to 40 change nothing but the loss's factor: ties, rows
    without experts, with too few of them, with NaN, infinities and lowest values."""
    inf, nan, low = float("inf"), float("nan"), torch.finfo(torch.float32).min
    g = torch.Generator().manual_seed(E)
    x = torch.randint(-2, 3, (400, E), generator=g).float()
    x[5] = -inf
    x[6, 2:] = -inf
    x[7, 1], x[8, 3], x[9, 0], x[10] = nan, inf, low, low
    x[11], x[12, 0], x[13, 2] = nan, -inf, 1e30
    x[12, 1:] = nan
    x = x.cuda()
    wide = torch.full((400, 40), -inf, device="cuda")
    wide[:, :E] = x
    mask = torch.rand(400, generator=g).cuda() > 0.1
    mask[5:14] = True
    a, b = (mxq.moe_route(t, k, mask=mask, renorm=renorm) for t in (x, wide))
    assert torch.equal(a.ids, b.ids) and torch.equal(a.counts, b.counts[:E]) and torch.equal(a.routed, b.routed)
    torch.testing.assert_close(a.weights, b.weights, rtol=2.0**-19, atol=0, equal_nan=True)
    assert a.loss.isnan() and b.loss.isnan()
    ok = ~x.isnan().any(1) & ~(x == inf).any(1)
    a, b = (mxq.moe_route(t, k, mask=mask & ok, renorm=renorm) for t in (x, wide))
    assert float(a.loss) == pytest.approx(float(b.loss) * E / 40, rel=2.0**-18)
    dw, dl = torch.randn(400, k, generator=g).cuda(), torch.tensor(0.3, device="cuda")
    da = mxq.moe_route_backward(x, a, dw, dl, mask=mask & ok, renorm=renorm)
    db = mxq.moe_route_backward(wide, b, dw, dl * E / 40, mask=mask & ok, renorm=renorm)
    torch.testing.assert_close(da, db[:, :E], rtol=2.0**-18, atol=2.0**-18 * 5)
    assert (da[~(mask & ok)] == 0).all()


@pytest.mark.parametrize("T,V,D,pad", [
    (16385, 16385, 8, 0), (20000, 3, 1001, 2), (30011, 20000, 33, 0), (40000, 40001, 16, 0), (17000, 64, 130, 1), (17000, 65, 24, 0),
])
@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
def test_rows_without_tokens_are_zero(T, V, D, pad, kind):
    """Many tokens, rows and runs of rows that none has; the rest exact sums, and
    nothing written beside the rows."""
    g = np.random.Generator(np.random.PCG64(T + V))
    live = np.sort(g.choice(V, max(1, V // 3), replace=False))
    ids = torch.from_numpy(live[g.integers(0, live.size, T)]).cuda()
    ids[:3] = torch.tensor([-1, V, 2**40])
    dy = torch.randint(-2, 3, (T, D), device="cuda").to(kind)
    room = torch.full((V, D + pad), 7.0, dtype=torch.float32, device="cuda")
    mxq.embedding_backward(ids, dy, V, out=room[:, :D])
    assert mxq.device_status(clear=True) == mxq.DEV_BADINDEX
    want = torch.zeros(V, D, dtype=torch.float64, device="cuda").index_add_(0, ids[3:], dy[3:].double())
    assert torch.equal(room[:, :D].double(), want) and (room[:, D:] == 7).all()
