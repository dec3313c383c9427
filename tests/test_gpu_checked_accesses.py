"""Which accesses of the training operators the checked library tests.

A watched address counts as outside its buffer: a call that touches it must report
DEV_OOB and leave it as it is.  For every buffer of every call the first and the last
element are watched in turn (inputs, outputs and the parts of the workspaces, whose
layouts are restated here), and the bytes around it, which no call may touch.  What a
call computes without the element is not looked at.  Tensor copies have their own
bounds (the tensor maps'), and single values at a given address are not computed.
"""
import pytest
import torch

import mx_block_quantization_gb300 as mxq
from mx_block_quantization_gb300 import training
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu
ALIGN = 256


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    if not mxq.debug_bounds():
        pytest.skip("the checked library's (the suite runs on it as well)")
    yield
    mxq.selftest_watch(0)
    mxq.device_status(clear=True)


def room(shape, dtype=torch.float32, pad=0, fill=None):
    """A matrix with `pad` elements between its rows, and bytes of its own on both sides."""
    *lead, n = shape
    count = 1
    for v in lead:
        count *= v
    es = torch.empty((), dtype=dtype).element_size()
    whole = torch.zeros(2 * ALIGN + (count * (n + pad) + 64) * es, dtype=torch.uint8, device="cuda")
    t = whole[ALIGN:ALIGN + count * (n + pad) * es].view(dtype).view(*lead, n + pad)[..., :n]
    if fill is not None:
        t.copy_(fill.to(dtype))
    return t


def ends(t):
    """Addresses of the first and the last element, and of bytes that are not the tensor's."""
    es = t.element_size()
    last = t.data_ptr() + sum((n - 1) * s for n, s in zip(t.shape, t.stride())) * es
    outside = [t.data_ptr() - es, last + es]
    if t.dim() > 1 and t.shape[-2] > 1 and t.stride(-2) > t.shape[-1]:
        outside.append(t.data_ptr() + t.shape[-1] * es)
    return [t.data_ptr(), last], outside


def reported(call, address):
    mxq.device_status(clear=True)
    mxq.selftest_watch(address)
    call()
    torch.cuda.synchronize()
    status = mxq.device_status(clear=True)
    mxq.selftest_watch(0)
    return bool(status & mxq.DEV_OOB)


class Workspace:
    """Stands in for the module's workspaces: one buffer at a known address."""

    def __init__(self, monkeypatch):
        self.room = torch.zeros(1 << 28, dtype=torch.uint8, device="cuda")
        self.bytes = 0
        monkeypatch.setattr(training, "_workspace", self.give)

    def give(self, size, what, device):
        assert 0 <= size <= self.room.numel(), what
        self.bytes = size
        return self.room, self.room.data_ptr() + ALIGN

    def at(self, offset):
        return self.room.data_ptr() + ALIGN + offset


def check(call, tensors, workspace=None, offsets=()):
    assert not reported(call, 0)
    missing = []
    for name, t in tensors.items():
        inside, outside = ends(t)
        for where, address in zip(("first", "last"), inside):
            before = t.clone()
            if not reported(call, address):
                missing.append((name, where))
            t.copy_(before)
        missing += [(name, "outside", a - t.data_ptr()) for a in outside if reported(call, a)]
    for name, offset in offsets:
        if not reported(call, workspace.at(offset)):
            missing.append(("workspace", name, offset))
    if workspace is not None and any(reported(call, workspace.at(o)) for o in (-4, workspace.bytes)):
        missing.append(("workspace", "outside"))
    assert not missing, missing


def up(n, to=256):
    return -(-n // to) * to


F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("kind", [F32, BF16])
@pytest.mark.parametrize("T,E,k,pad", [(300, 8, 2, 1), (20, 30, 3, 0), (200, 40, 4, 3), (77, 256, 8, 0), (40, 600, 5, 0)])
def test_routing(monkeypatch, T, E, k, pad, kind):
    ws = Workspace(monkeypatch)
    x = room((T, E), kind, pad, torch.randn(T, E, device="cuda"))
    mask = room((T,), torch.uint8, fill=torch.ones(T))
    out = mxq.Routing(room((T, k)), room((T, k), torch.int32), room((E,), torch.int32), torch.zeros((), device="cuda"),
                      torch.zeros((), dtype=torch.int32, device="cuda"))
    at_once = 128 if E <= 32 else 32 if E <= 256 else 16 if E <= 512 else 8
    blocks = -(-T // at_once)
    parts = []
    if blocks > 1:
        c, n, loss = 4 * blocks * E, 8 * blocks * E, 8 * blocks * E + 4 * blocks + 4
        parts = [("p", 0), ("p", c - 4), ("c", c), ("c", n - 4), ("n", n), ("n", n + 4 * blocks - 4), ("loss", loss),
                 ("loss", loss + 4 * (-(-E // 32) - 1))]
    check(lambda: mxq.moe_route(x, k, mask=mask, out=out),
          dict(logits=x, mask=mask, weights=out.weights, ids=out.ids, counts=out.counts), ws, parts)
    mxq.moe_route(x, k, mask=mask, out=out)
    dw, dl = room((T, k), fill=torch.randn(T, k, device="cuda")), torch.ones((), device="cuda")
    dx = room((T, E), kind, pad)
    check(lambda: mxq.moe_route_backward(x, out, dw, dl, mask=mask, out=dx),
          dict(logits=x, mask=mask, ids=out.ids, counts=out.counts, dweights=dw, dlogits=dx))


@pytest.mark.parametrize("kind", [F32, BF16])
@pytest.mark.parametrize("T,E,k,D,pad", [(20, 3, 2, 64, 0), (700, 5, 4, 40, 8), (30, 4, 3, 33, 1), (300, 3, 8, 2050, 0),
                                         (30, 12, 10, 2048, 0), (7000, 3, 2, 16, 0)])
def test_exchange(monkeypatch, T, E, k, D, pad, kind):
    ws = Workspace(monkeypatch)
    k = min(k, E)
    ids = room((T, k), torch.int32, fill=torch.rand(T, E, device="cuda").argsort(1)[:, :k])
    M = mxq.moe_rows(T, k, E) + 128        # the last rows belong to no group
    plan = mxq.MoePlan(room((E,), torch.int32), room((T, k), torch.int32), room((M,), torch.int32))
    chunks = -(-T * k // 1024)
    check(lambda: mxq.moe_plan(ids, E, out=plan),
          dict(ids=ids, offs=plan.offs, slots=plan.slots, source=plan.source), ws,
          [("counts", 0), ("counts", 4 * chunks * E - 4)] if chunks > 1 else [])
    mxq.moe_plan(ids, E, out=plan)
    x, rows = room((T, D), kind, pad, torch.randn(T, D, device="cuda")), room((M, D), kind, pad)
    plan_of = dict(slots=plan.slots, source=plan.source)
    check(lambda: mxq.moe_dispatch(x, plan, out=rows), dict(x=x, rows=rows, **plan_of))
    # the last row that a token takes, for the calls that read rows
    used = int((plan.source >= 0).nonzero()[-1]) + 1
    w, y = room((T, k), fill=torch.rand(T, k, device="cuda")), room((T, D), kind, pad)
    few = rows[:used]
    for weights in (w, None):
        tensors = dict(y=y, slots=plan.slots)
        if weights is not None:
            tensors["weights"] = w
        call = lambda: mxq.moe_combine(rows, plan, weights, out=y)
        check(call, tensors)
        assert all(reported(call, a) for a in ends(few)[0])
    drows, dweights = room((M, D), kind, pad), room((T, k))
    call = lambda: mxq.moe_combine_backward(x, rows, plan, w, out=(drows, dweights))
    check(call, dict(dy=x, drows=drows, dweights=dweights, weights=w, **plan_of))
    assert all(reported(call, a) for a in ends(few)[0])


@pytest.mark.parametrize("kind", [F32, BF16])
@pytest.mark.parametrize("ids_type", [torch.int32, torch.int64])
@pytest.mark.parametrize("T,V,D,pad", [(9, 50, 64, 0), (300, 70, 33, 2), (20000, 300, 40, 0), (20000, 30000, 17, 1), (70000, 6, 16, 0),
                                       (1100, 5000, 8, 0)])
def test_embedding(monkeypatch, T, V, D, pad, ids_type, kind):
    ws = Workspace(monkeypatch)
    ids = torch.randint(0, V, (T,), device="cuda")
    ids[0], ids[-1] = 0, V - 1
    ids = room((T,), ids_type, fill=ids)
    table = room((V, D), kind, pad, torch.randn(V, D, device="cuda"))
    y = room((T, D), kind, pad, torch.randn(T, D, device="cuda"))
    check(lambda: mxq.embedding(ids, table, out=y), dict(ids=ids, table=table, y=y))
    grad = room((V, D), kind, pad)
    small = T <= 16384
    bits = V.bit_length()
    passes = -(-bits // 10)
    digit = -(-bits // passes)
    chunks = min(128, -(-T // 1024))
    per = up(-(-T // chunks), 1024)
    chunks = -(-T // per)
    keys = up(4 * (chunks << digit))
    parts = [] if small else [("counts", 0), ("counts", 4 * (chunks << digit) - 4)]
    last = 0 if small else 8 * T * ((passes - 1) & 1)       # the buffer of the last pass
    parts += [("keys", keys + last), ("keys", keys + last + 4 * T - 4), ("tokens", keys + last + 4 * T),
              ("tokens", keys + last + 8 * T - 4)]
    call = lambda: mxq.embedding_backward(ids, y, V, out=grad)
    check(call, dict(ids=ids, dy=y, dtable=grad), ws, parts)
    if T > 32:                                              # one long run: a piece per 32 places
        ids.fill_(V - 1)
        pieces = keys + up(16 * T)
        end = pieces + 4 * (2 * (-(-T // 32) - 1) * D + D)
        check(call, dict(ids=ids, dtable=grad), ws, [("pieces", pieces), ("pieces", pieces + 4 * D - 4), ("pieces", end - 4)])


def ortho_parts(batch, m, n):
    """Offsets of the workspace's parts that the kernels reach without tensor maps."""
    side, long = min(m, n), max(m, n)
    ldx, lds, parts = up(n, 8), up(side, 8), 2 if side <= 64 else 1
    xb, sb = up(batch * m * ldx * 2), up(batch * side * lds * 2)
    at = parts * (2 * xb + 2 * sb)
    d_gram, d_poly = at, at + up(batch * lds * 4)
    sums = d_poly + up(batch * lds * 4)
    lifts = sums + up(batch * 2048 * 12)
    partial = lifts + up(batch * 4)
    x_end = 2 * ((batch - 1) * m * ldx + (m - 1) * ldx + n)
    found = [("x", 0), ("x", x_end - 2), ("sums", sums), ("sums", sums + 8), ("lifts", lifts), ("lifts", lifts + 4 * batch - 4)]
    if parts == 2:
        low = 2 * xb + 2 * sb
        found += [("x low", low), ("x low", low + x_end - 2)]
    else:
        for name, d in (("d_gram", d_gram), ("d_poly", d_poly)):
            found += [(name, d), (name, d + 4 * ((batch - 1) * lds + side) - 4)]
    return found, partial, batch * side * lds * 4, 2 * xb, sb, lds


@pytest.mark.parametrize("kind", [F32, BF16])
@pytest.mark.parametrize("batch,m,n,pad", [(1, 20, 30, 0), (2, 50, 33, 3), (1, 130, 200, 0), (2, 200, 130, 8), (1, 300, 5000, 0),
                                           (1, 40, 9000, 0), (1, 5001, 300, 1)])
def test_orthogonalize(monkeypatch, batch, m, n, pad, kind):
    ws = Workspace(monkeypatch)
    g = room((batch, m, n), kind, pad, torch.randn(batch, m, n, device="cuda"))
    out = room((batch, m, n), BF16, pad=pad | 1)            # no tensor map takes an odd pitch
    found, partial, square, gram, sb, lds = ortho_parts(batch, m, n)
    call = lambda: mxq.orthogonalize(g, out=out, steps=2)
    call()
    if ws.bytes > partial:                                  # K in slices
        slices = (ws.bytes - partial) // square
        assert slices >= 2
        found += [("partial", partial), ("partial", partial + square - 4), ("partial", partial + square)]
        found += [("gram", gram), ("gram", gram + 2 * ((batch * min(m, n) - 1) * lds + min(m, n)) - 2)]
        if min(m, n) <= 64:
            low = gram + 2 * sb + gram
            found += [("gram low", low), ("gram low", low + 2 * ((batch * min(m, n) - 1) * lds + min(m, n)) - 2)]
    check(call, dict(g=g, out=out), ws, found)
    # the diagonals' remainders where the polynomial takes an addend
    if min(m, n) > 64:
        plain = lambda: mxq.orthogonalize(g, out=out, steps=1, coefficients=(1.5, -0.5, 0.0))
        check(plain, dict(g=g), ws, [f for f in found if f[0] in ("d_gram", "d_poly")])
