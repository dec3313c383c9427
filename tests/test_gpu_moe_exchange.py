"""The exchange of rows with the expert groups against its definition.

Plan and dispatch are exact.  Sums over at most 32 choices in fp32 are held to
k units of 2^-24 of the sum of magnitudes, plus half a unit of bf16 where the
result is rounded to it; the dot products of dweights, whose D products are added
by up to 256 threads, to (D/256 + 20) units of theirs.
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


def plan_of(ids, experts, M):
    flat = ids.reshape(-1)
    offs, slots, source = [], np.full(flat.size, -1), np.full(M, -1)
    row = 0
    for e in range(experts):
        own = np.flatnonzero(flat == e)
        slots[own] = row + np.arange(own.size)
        source[row:row + own.size] = own
        row += -(-own.size // 128) * 128
        offs.append(row)
    return np.array(offs), slots.reshape(ids.shape), source


def routing(T, E, k, seed=0, dropped=0.1, skew=2.0):
    g = np.random.Generator(np.random.PCG64(seed + 31 * T + E))
    liked = g.normal(size=E) * skew
    ids = np.argsort(-(g.normal(size=(T, E)) + liked), axis=1)[:, :k].astype(np.int32)
    ids[g.random(T) < dropped] = -1
    return ids


def check_plan(ids, E, rows=None):
    T, k = ids.shape
    plan = mxq.moe_plan(torch.from_numpy(ids).cuda(), E, rows=rows)
    M = plan.source.numel()
    offs, slots, source = plan_of(ids, E, M)
    assert M % 128 == 0 and M >= offs[-1]
    assert np.array_equal(plan.offs.cpu().numpy(), offs)
    assert np.array_equal(plan.slots.cpu().numpy(), slots)
    assert np.array_equal(plan.source.cpu().numpy(), source)
    return plan, slots, source


@pytest.mark.parametrize("T,E,k", [
    (1, 1, 1), (1, 64, 8), (2, 3, 2), (31, 5, 1), (128, 1, 1), (129, 2, 2), (255, 7, 4), (512, 16, 2), (513, 16, 2),
    (1000, 256, 8), (3000, 1024, 3), (7168, 64, 8), (40000, 100, 6), (70001, 33, 2),
])
def test_plan(T, E, k):
    check_plan(routing(T, E, k), E)


def test_plan_extremes():
    check_plan(np.zeros((5000, 1), np.int32), 9)                       # one expert takes all
    check_plan(np.full((5000, 2), 8, np.int32), 9)                     # the last one, twice a token
    check_plan(np.full((300, 2), -1, np.int32), 4)                     # nobody is routed
    check_plan(np.arange(1024, dtype=np.int32).reshape(1024, 1), 1024)  # one token each: mostly padding
    check_plan(routing(100, 8, 2), 8, rows=4096)                       # more rows than needed
    assert mxq.moe_rows(7168, 8, 64) == 65408 and mxq.moe_rows(1, 1, 64) == 128 and mxq.moe_rows(0, 1, 64) == 0
    p = mxq.moe_plan(torch.empty(0, 4, dtype=torch.int32, device="cuda"), 6)
    assert p.offs.tolist() == [0] * 6 and p.source.numel() == 0 and p.slots.shape == (0, 4)


def test_plan_leaves_out_ids_out_of_range_and_says_so():
    ids = routing(400, 8, 3, dropped=0)
    bad = ids.copy()
    bad[5, 1], bad[399, 2], bad[0, 0] = 8, -2, 2**31 - 1
    got = mxq.moe_plan(torch.from_numpy(bad).cuda(), 8)
    assert mxq.device_status(clear=True) == mxq.DEV_BADINDEX
    bad[(bad < 0) | (bad >= 8)] = -1
    want = plan_of(bad, 8, got.source.numel())
    for a, b in zip(got, want):
        assert np.array_equal(a.cpu().numpy(), b)


def matrix(rows, D, kind, pad=0, seed=0):
    g = torch.Generator().manual_seed(seed + rows * 7 + D)
    return torch.randn(rows, D + pad, generator=g).to(TYPES[kind]).cuda()[:, :D]


def half_unit(kind, want):
    return 2.0**-8 * np.abs(want) if kind == "bf16" else 0.0


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("T,D,E,k,pad", [
    (1, 1, 1, 1, 0), (1, 64, 64, 8, 0), (3, 7, 4, 2, 0), (17, 33, 5, 3, 3), (64, 130, 9, 2, 0), (50, 256, 8, 8, 8),
    (33, 1024, 16, 4, 0), (130, 1001, 6, 3, 0), (20, 2050, 12, 9, 0), (9, 4100, 3, 3, 4), (300, 96, 40, 32, 0),
    (700, 2048, 64, 8, 0),
])
def test_rows(T, D, E, k, pad, kind):
    ids = routing(T, E, k)
    plan, slots, source = check_plan(ids, E)
    M = source.size
    x, h, dy = matrix(T, D, kind, pad), matrix(M, D, kind, pad, 1), matrix(T, D, kind, pad, 2)
    w = torch.rand(T, k, generator=torch.Generator().manual_seed(4)).cuda()

    rows = mxq.moe_dispatch(x, plan)
    want = torch.zeros_like(rows)
    live = torch.from_numpy(np.flatnonzero(source >= 0)).cuda()
    want[live] = x[torch.from_numpy(source[source >= 0] // k).cuda()]
    assert torch.equal(rows, want)

    h64, dy64, w64 = (t.double().cpu().numpy() for t in (h, dy, w))
    picked = np.where((slots >= 0)[..., None], h64[np.maximum(slots, 0)], 0.0)   # [T, k, D]
    unit = (k + 1) * 2.0**-24
    for weights, f in ((w, w64), (None, np.ones_like(w64))):
        got = mxq.moe_combine(h, plan, weights).double().cpu().numpy()
        y = np.einsum("tk,tkd->td", f, picked)
        size = np.einsum("tk,tkd->td", np.abs(f), np.abs(picked))
        assert (np.abs(got - y) <= unit * size + half_unit(kind, y)).all()

    drows, dweights = mxq.moe_combine_backward(dy, h, plan, w)
    dr = np.zeros((M, D))
    dr[source >= 0] = w64.reshape(-1)[source[source >= 0], None] * dy64[source[source >= 0] // k]
    assert (np.abs(drows.double().cpu().numpy() - dr) <= 2.0**-24 * np.abs(dr) + half_unit(kind, dr)).all()
    assert (drows.cpu()[torch.from_numpy(source < 0)] == 0).all()
    dot = np.einsum("td,tkd->tk", dy64, picked)
    size = np.einsum("td,tkd->tk", np.abs(dy64), np.abs(picked))
    assert (np.abs(dweights.double().cpu().numpy() - dot) <= (D / 256 + 20) * 2.0**-24 * size + 1e-37).all()
    assert (dweights.cpu()[torch.from_numpy(slots < 0)] == 0).all()


def test_gradient_of_dispatch_is_combine_without_weights():
    """<dispatch(x), g> = <x, combine(g)> for every x and g: exact in fp32 for small
    whole numbers."""
    ids = routing(90, 12, 4)
    plan = mxq.moe_plan(torch.from_numpy(ids).cuda(), 12)
    g = torch.Generator().manual_seed(1)
    x = torch.randint(-8, 9, (90, 40), generator=g).float().cuda()
    r = torch.randint(-8, 9, (plan.source.numel(), 40), generator=g).float().cuda()
    assert (mxq.moe_dispatch(x, plan).double() * r.double()).sum() == (x.double() * mxq.moe_combine(r, plan).double()).sum()


def test_combine_gradients_against_differences():
    """<combine(h + eps d, w + eps v) - combine(h - eps d, w - eps v), dy> / 2 eps: the
    function is of second degree, so central differences in 64 bits are exact."""
    T, k, E, D = 40, 3, 6, 24
    ids = routing(T, E, k)
    plan, slots, source = check_plan(ids, E)
    M = source.size
    h, d, dy = matrix(M, D, "f32", seed=1), matrix(M, D, "f32", seed=2), matrix(T, D, "f32", seed=3)
    w, v = matrix(T, k, "f32", seed=4), matrix(T, k, "f32", seed=5)
    drows, dweights = mxq.moe_combine_backward(dy, h, plan, w.contiguous())

    def combine(hh, ww):
        picked = torch.where((plan.slots >= 0)[..., None], hh[plan.slots.clamp(min=0).long()], 0.0)
        return (ww[..., None] * picked).sum(1)
    up = combine(h.double() + d.double(), w.double() + v.double())
    down = combine(h.double() - d.double(), w.double() - v.double())
    want = ((up - down) / 2 * dy.double()).sum()
    got = (drows.double() * d.double()).sum() + (dweights.double() * v.double()).sum()
    assert float(got) == pytest.approx(float(want), rel=1e-4, abs=1e-3)


def test_the_grouped_cast_takes_the_dispatched_rows():
    """rows and offs go into the dual-axis cast as they are, and its unused tail
    has zero column scales."""
    T, k, E, D = 300, 2, 6, 256
    plan = mxq.moe_plan(torch.from_numpy(routing(T, E, k)).cuda(), E, rows=2048)
    rows = mxq.moe_dispatch(matrix(T, D, "bf16"), plan)
    out = mxq.quantize_2d_dual(rows, plan.offs)
    torch.cuda.synchronize()
    assert mxq.device_status(clear=True) == 0
    end = int(plan.offs[-1])
    assert (out.s_col[D * end // 32:] == 0).all() and (out.q_row[end:] == 0).all()


def test_strided_outputs_streams_and_no_rows():
    T, k, E, D = 60, 2, 5, 48
    plan = mxq.moe_plan(torch.from_numpy(routing(T, E, k)).cuda(), E)
    M = plan.source.numel()
    x, h = matrix(T, D, "bf16"), matrix(M, D, "bf16", seed=1)
    wide = torch.full((M, D + 5), 2.0, dtype=torch.bfloat16, device="cuda")
    mxq.moe_dispatch(x, plan, out=wide[:, :D])
    assert torch.equal(wide[:, :D], mxq.moe_dispatch(x, plan)) and (wide[:, D:] == 2).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = mxq.moe_combine(h, plan, stream=side)
    side.synchronize()
    assert torch.equal(y, mxq.moe_combine(h, plan))
    none = mxq.moe_plan(torch.empty(0, k, dtype=torch.int32, device="cuda"), E, rows=256)
    assert (mxq.moe_dispatch(x[:0], none) == 0).all()
    assert mxq.moe_combine(h[:256], none).shape == (0, D)
    drows, dweights = mxq.moe_combine_backward(x[:0], h[:256], none, torch.empty(0, k, device="cuda"))
    assert (drows == 0).all() and dweights.shape == (0, k)


def test_slots_out_of_range_are_left_out():
    T, k, E, D = 20, 2, 3, 16
    plan = mxq.moe_plan(torch.from_numpy(routing(T, E, k, dropped=0)).cuda(), E)
    M = plan.source.numel()
    h = matrix(M, D, "f32")
    slots = plan.slots.clone()
    slots[3, 1], slots[4, 0] = M, -5
    y = mxq.moe_combine(h, mxq.MoePlan(plan.offs, slots, plan.source))
    assert mxq.device_status(clear=True) == mxq.DEV_BADINDEX
    assert torch.equal(y[3], h[slots[3, 0].item()]) and torch.equal(y[4], h[slots[4, 1].item()])


def test_refusals():
    ids = torch.from_numpy(routing(10, 4, 2)).cuda()
    plan = mxq.moe_plan(ids, 4)
    M = plan.source.numel()
    x = matrix(10, 8, "f32")
    for bad in (ids.long(), ids.cpu(), ids[0], ids.t()):
        with pytest.raises(ValueError):
            mxq.moe_plan(bad, 4)
    for rows in (0, 100, M - 128, M + 1):
        with pytest.raises(mxq.MxqError):
            mxq.moe_plan(ids, 4, rows=rows)
    with pytest.raises(mxq.MxqError):
        mxq.moe_plan(ids, 1025)
    with pytest.raises(mxq.MxqError):
        mxq.moe_plan(torch.zeros(4, 33, dtype=torch.int32, device="cuda"), 4)
    for bad in (x[:9], x.half(), x.cpu(), matrix(8, 10, "f32").t()):
        with pytest.raises(ValueError):
            mxq.moe_dispatch(bad, plan)
    h = matrix(M, 8, "f32")
    with pytest.raises(ValueError):
        mxq.moe_combine(h[:-1], plan)
    with pytest.raises(ValueError):
        mxq.moe_combine(h, plan, torch.zeros(10, 3, device="cuda"))
    with pytest.raises(ValueError):
        mxq.moe_combine_backward(x.bfloat16(), h, plan, torch.zeros(10, 2, device="cuda"))
    with pytest.raises(mxq.MxqError) as e:
        mxq.moe_combine(h, plan, out=h[:10])
    assert e.value.code == mxq.EOVERLAP
