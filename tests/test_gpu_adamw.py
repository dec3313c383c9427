"""adamw_step against its formula in 64 bits, and its bytes against a restatement.

Tolerances, in units of 2^-24: g one rounding (the scale); m three (two products, one
sum) of the terms' sizes; v four.  The update divides m by a root and an epsilon that are
right to 8 units (root, reciprocal, product and sum, the approximate division's 2 of
2^-23) times a rate that is right to 8 (expm1, its argument, division); and m's own error.
p adds three roundings of its size, and half a step of bf16 where it is one.
In 8 bits m and the root are rounded to fp32 as the formulas stand, which numpy does the
same way, so the bytes are equal.
"""
import math

import numpy as np
import pytest
import torch

import mx_block_quantization_gb300 as mxq
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
U = 2.0**-24
HOW = dict(lr=1e-2, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    yield
    torch.cuda.empty_cache()
    assert mxq.device_status(clear=True) == 0


def tensors(sizes, dtype=F32, at=0, scale=1.0, seed=0):
    """Tensors that begin `at` elements behind an aligned address."""
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(n + at, generator=g) * scale).to(dtype).cuda()[at:] for n in sizes]


def starts_of(sizes):
    at = np.concatenate([[0], np.cumsum([-(-n // 128) * 128 for n in sizes])])
    return at[:-1].tolist()


def wanted(p, g, m, v, t, scale, lr, betas, eps, weight_decay):
    """p, m, v after the step and how far they may be off, in 64 bits."""
    b1, b2 = betas
    g = g * scale
    m1, v1 = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
    m_off = 4 * U * (abs(b1 * m) + abs((1 - b1) * g))
    v_off = 6 * U * v1
    rate, denom = lr / (1 - b1**t), (v1 / (1 - b2**t)).sqrt() + eps
    update = rate * m1 / denom
    p1 = p * (1 - lr * weight_decay) - update
    p_off = rate * m_off / denom + 24 * U * update.abs() + 3 * U * (p.abs() + p1.abs())
    return p1, m1, v1, p_off, m_off, v_off


SIZES = [1, 31, 32, 33, 0, 127, 128, 129, 4095, 4096, 4097, 8191, 100003]


@pytest.mark.parametrize("kind", [F32, BF16])
@pytest.mark.parametrize("gkind", [F32, BF16])
@pytest.mark.parametrize("at", [0, 1, 2])
def test_steps_in_32_bits(kind, gkind, at):
    params = tensors(SIZES, kind, at)
    copies = [torch.empty_like(p, dtype=BF16) for p in params]
    copies[3] = None
    moments = mxq.adamw_moments(params)
    scale = torch.tensor(0.37, device="cuda")
    for t in (1, 2, 3):
        grads = tensors(SIZES, gkind, at, 0.1, seed=t)
        before = [p.double() for p in params], moments.m.double(), moments.v.double()
        mxq.adamw_step(params, grads, moments, t, grad_scale=scale, copies=copies, **HOW)
        for i, (p, g, lo, n) in enumerate(zip(params, grads, starts_of(SIZES), SIZES)):
            p1, m1, v1, p_off, m_off, v_off = wanted(before[0][i], g.double(), before[1][lo:lo + n], before[2][lo:lo + n], t,
                                                     float(scale), **HOW)
            if kind == BF16:
                p_off = p_off + 2.0**-8 * (p1.abs() + p_off)
            assert bool(((p.double() - p1).abs() <= p_off).all())
            assert bool(((moments.m[lo:lo + n].double() - m1).abs() <= m_off).all())
            assert bool(((moments.v[lo:lo + n].double() - v1).abs() <= v_off).all())
            assert not moments.m[lo + n:lo + -(-n // 128) * 128].any()
            if copies[i] is not None:
                assert torch.equal(copies[i], p.to(BF16)) or kind == BF16 and torch.equal(copies[i], p)


def mixed(x):
    x = np.uint32(x)
    with np.errstate(over="ignore"):
        x = x ^ (x >> np.uint32(16))
        x = x * np.uint32(0x6A09E667)
        x = x ^ (x >> np.uint32(15))
        x = x * np.uint32(0xBB67AE85)
    return x ^ (x >> np.uint32(16))


def random_bits(seed, t, place):
    key = mixed(mixed(mixed(np.uint32(seed & 0xFFFFFFFF)) ^ np.uint32(seed >> 32)) ^ np.uint32(t))
    return mixed(place.astype(np.uint32) ^ key ^ mixed((place >> 32).astype(np.uint32)))


E4M3 = np.array([((b & 7) * 2.0**-9 if b >> 3 & 15 == 0 else (8 + (b & 7)) * 2.0**((b >> 3 & 15) - 10)) for b in range(127)])


def encode(x, u, keep):
    """Bytes and scales of x [blocks, 32] (64 bits), rounded up where the part of the way to
    the next value is at least 1 - u."""
    most = np.abs(x).max(1)
    with np.errstate(divide="ignore"):
        s = np.where(most > 0, np.maximum(np.ceil(np.log2(np.maximum(most, 1e-300) / 448)), -127), -127)
    a = np.abs(x) * 2.0**-s[:, None]
    low = np.searchsorted(E4M3, a, side="right") - 1
    gap = np.where(low < 126, E4M3[np.minimum(low + 1, 126)] - E4M3[low], 1.0)
    code = np.minimum(low + ((a - E4M3[low]) / gap + u >= 1), 126)
    if keep:
        code = np.where((x != 0) & (code == 0), 1, code)
    return np.where(np.signbit(x), code | 128, code).astype(np.uint8), (s + 127).astype(np.uint8)


def decode(q, s):
    v = E4M3[np.minimum(q & 127, 126)] * np.where(q & 128, -1.0, 1.0)
    return v * np.repeat(2.0**(s.astype(np.float64) - 127), 32)


@pytest.mark.parametrize("at,kind,gkind", [(0, F32, F32), (1, F32, BF16), (0, BF16, BF16), (3, BF16, F32)])
def test_steps_in_8_bits(at, kind, gkind):
    params = tensors(SIZES, kind, at)
    moments = mxq.adamw_moments(params, 8)
    total, seed = moments.m.numel(), 0x123456789ABCDEF0
    f = np.float32
    b1, b2 = HOW["betas"]
    for t in (1, 2, 3, 4):
        grads = tensors(SIZES, gkind, at, 0.1, seed=t)
        for g in grads:
            g[::7] *= 1e-5
            g[::11] = 0
        before = [p.double() for p in params], [x.cpu().numpy() for x in moments]
        m0, r0 = decode(before[1][0], before[1][2]), decode(before[1][1], before[1][3])
        mxq.adamw_step(params, grads, moments, t, seed=seed, **HOW)
        after = [x.cpu().numpy() for x in moments]
        for p, b, g, lo, n in zip(params, before[0], grads, starts_of(SIZES), SIZES):
            if n == 0:
                continue
            m, r, g = m0[lo:lo + n], r0[lo:lo + n], g.cpu().float().numpy()
            dev = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
            p1, _, _, p_off, _, _ = wanted(b, dev(g).double(), dev(m), dev(r * r), t, 1.0, **HOW)
            if kind == BF16:
                p_off = p_off + 2.0**-8 * (p1.abs() + p_off)
            assert bool(((p.double() - p1).abs() <= p_off).all())
            m32, r32 = m.astype(f), r.astype(f)
            m1 = f(b1) * m32 + f(1 - b1) * g
            root = np.sqrt(f(b2) * (r32 * r32) + f(1 - b2) * (g * g))
            blocks = -(-n // 32)
            pad = lambda x: np.pad(x.astype(np.float64), (0, 32 * blocks - n)).reshape(-1, 32)  # noqa: E731
            bits = random_bits(seed, t, lo + np.arange(32 * blocks, dtype=np.int64)).reshape(-1, 32)
            for x, u, q, s, keep in ((m1, bits & 0xFFFF, 0, 2, False), (root, bits >> 16, 1, 3, True)):
                want_q, want_s = encode(pad(x), u / 65536, keep)
                assert np.array_equal(after[s][lo // 32:lo // 32 + blocks], want_s)
                got = after[q][lo:lo + 32 * blocks]
                # a zero has no sign that counts
                assert np.array_equal(np.where(got & 127, got, 0), np.where(want_q & 127, want_q, 0).reshape(-1))
            end = -(-n // 128) * 128
            assert not after[0][lo + 32 * blocks:lo + end].any() and not after[1][lo + 32 * blocks:lo + end].any()
    assert total == moments.m.numel()


def test_the_mean_of_the_rounding_is_the_value():
    """Over 4096 steps' seeds the mean of n draws of a value between two neighbours is off
    by at most five of its deviations, half a gap / sqrt(n), and the random bits' 2^-17."""
    n = 32 * 40
    g = tensors([n], scale=1.0, seed=3)
    zero = torch.zeros(n, device="cuda")
    sums = [torch.zeros(n, dtype=torch.float64, device="cuda") for _ in range(2)]
    rounds = 4096
    for seed in range(rounds):
        moments = mxq.adamw_moments(g, 8)
        mxq.adamw_step([zero], g, moments, 1, seed=seed * 0x9E3779B97F4A7C15 % 2**64, **HOW)
        for acc, q, s in ((sums[0], moments.m, moments.m_scale), (sums[1], moments.v, moments.v_scale)):
            acc += q.view(torch.float8_e4m3fn).double() * torch.exp2(s.double() - 127).repeat_interleave(32)
    m = 0.1 * g[0].double()
    for acc, want in ((sums[0], m), (sums[1], (0.05 * g[0].double() ** 2).sqrt())):
        size = want.view(-1, 32).abs().amax(1).repeat_interleave(32)
        gap = torch.maximum(want.abs() / 8, size / 448 * 2**-9 * 2)
        sure = want.abs() > size * 2.0**-17          # the smallest roots are kept from 0
        off = (acc / rounds - want).abs()
        assert bool((off <= 5 * gap / 2 / math.sqrt(rounds) + gap * 2.0**-16)[sure].all())


def test_a_root_is_never_rounded_to_zero():
    g = torch.full((32,), 1e-9, device="cuda")
    g[0] = 1.0
    p = torch.zeros(32, device="cuda")
    moments = mxq.adamw_moments([p], 8)
    mxq.adamw_step([p], [g], moments, 1, **HOW)
    assert bool((moments.v[:32].view(torch.float8_e4m3fn).float() > 0).all())
    for t in range(2, 40):
        mxq.adamw_step([p], [torch.zeros_like(g)], moments, t, seed=t, **HOW)
    assert bool(torch.isfinite(p).all()) and float(p.abs().max()) < 1.0


def test_values_that_are_not_finite():
    g = torch.ones(96, device="cuda")
    g[40] = math.inf
    p = torch.zeros(96, device="cuda")
    moments = mxq.adamw_moments([p], 8)
    mxq.adamw_step([p], [g], moments, 1, **HOW)
    for q, s in ((moments.m, moments.m_scale), (moments.v, moments.v_scale)):
        assert s[:3].tolist()[1] == 255 and bool((q[32:64] == 0x7F).all())
        assert s[0] != 255 and s[2] != 255 and not bool((q[:32] == 0x7F).any())
    mxq.adamw_step([p], [torch.ones_like(g)], moments, 2, **HOW)
    nan = torch.isnan(p)
    assert bool(nan[32:64].all()) and not nan[:32].any() and not nan[64:].any()


@pytest.mark.parametrize("bits", [32, 8])
def test_gradients_of_none_leave_their_tensors(bits):
    params = tensors([100, 300, 5000])
    moments = mxq.adamw_moments(params, bits)
    mxq.adamw_step(params, tensors([100, 300, 5000], seed=1), moments, 1, **HOW)
    before = [p.clone() for p in params], [None if x is None else x.clone() for x in moments]
    grads = tensors([100, 300, 5000], seed=2)
    grads[1] = None
    mxq.adamw_step(params, grads, moments, 2, **HOW)
    assert torch.equal(params[1], before[0][1]) and not torch.equal(params[2], before[0][2])
    assert torch.equal(moments.m[128:512], before[1][0][128:512])
    assert not torch.equal(moments.m[512:], before[1][0][512:])
    mxq.adamw_step([], [], moments, 1, **HOW)
    mxq.adamw_step(params, [None] * 3, moments, 3, **HOW)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("count", [32, 33, 512, 1100])
def test_many_tensors(count, bits):
    """Both parameter lists, and more tensors than one launch takes: each as by itself."""
    sizes = [1 + 37 * i % 700 for i in range(count)]
    params, grads = tensors(sizes), tensors(sizes, seed=1)
    flat = torch.zeros(sum(-(-n // 128) * 128 for n in sizes), device="cuda")
    grad = torch.zeros_like(flat)
    for p, g, at in zip(params, grads, starts_of(sizes)):
        flat[at:at + p.numel()] = p
        grad[at:at + p.numel()] = g
    moments, whole = mxq.adamw_moments(params, bits), mxq.adamw_moments([flat], bits)
    for t in (1, 2):
        mxq.adamw_step(params, grads, moments, t, seed=5, **HOW)
        mxq.adamw_step([flat], [grad], whole, t, seed=5, **HOW)
    for p, at in zip(params, starts_of(sizes)):
        assert torch.equal(p, flat[at:at + p.numel()])
    assert torch.equal(moments.m, whole.m) and torch.equal(moments.v, whole.v)


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_and_replayed(bits):
    """Step and rate on the device: replays go on as eager calls do."""
    sizes = [1000, 77]
    eager, own = tensors(sizes), tensors(sizes)
    me, mo = mxq.adamw_moments(eager, bits), mxq.adamw_moments(own, bits)
    grads = tensors(sizes, seed=1)
    step, lr = torch.ones((), dtype=torch.int64, device="cuda"), torch.tensor(1e-2, device="cuda")
    how = {**HOW, "lr": lr}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        mxq.adamw_step(own, grads, mo, step, seed=3, **how)
        step += 1
    for t in (1, 2, 3, 4):
        lr.fill_(1e-2 / t)
        grads[0].normal_()
        graph.replay()
        mxq.adamw_step(eager, grads, me, torch.tensor(t, device="cuda"), seed=3, **how)
        assert all(torch.equal(a, b) for a, b in zip(own, eager))
        assert torch.equal(mo.m, me.m) and torch.equal(mo.v, me.v)
    # a number for the step is the same step
    a, b = tensors(sizes), tensors(sizes)
    ma, mb = mxq.adamw_moments(a, bits), mxq.adamw_moments(b, bits)
    mxq.adamw_step(a, grads, ma, 7, seed=3, **how)
    mxq.adamw_step(b, grads, mb, torch.tensor(7, device="cuda"), seed=3, **how)
    assert torch.equal(a[0], b[0]) and torch.equal(ma.m, mb.m) and torch.equal(ma.v, mb.v)


def test_on_a_stream_and_with_other_seeds():
    sizes = [5000]
    params = tensors(sizes)
    grads = tensors(sizes, seed=1)
    a, b, c = (mxq.adamw_moments(params, 8) for _ in range(3))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    mxq.adamw_step(params, grads, a, 1, seed=1, stream=side, **HOW)
    side.synchronize()
    mxq.adamw_step(tensors(sizes), grads, b, 1, seed=1, **HOW)
    mxq.adamw_step(tensors(sizes), grads, c, 1, seed=2, **HOW)
    assert torch.equal(a.m, b.m) and torch.equal(a.v, b.v) and torch.equal(a.m_scale, b.m_scale)
    assert not torch.equal(a.m, c.m) and torch.equal(a.m_scale, c.m_scale)


def test_moments_past_32_bits():
    """Places of moments past 2^32: the random bits take the high part, the bytes are where they belong."""
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    big = (1 << 32) + 128
    params = [torch.zeros(big, dtype=BF16, device="cuda"), torch.zeros(64, device="cuda")]
    grads = [None, torch.ones(64, device="cuda")]
    moments = mxq.adamw_moments(params, 8)
    mxq.adamw_step(params, grads, moments, 1, seed=9, **HOW)
    bits = random_bits(9, 1, big + np.arange(64, dtype=np.int64)).reshape(-1, 32)
    q, s = encode(np.full((2, 32), np.float64(np.float32(1 - HOW["betas"][0]))), (bits & 0xFFFF) / 65536, False)
    assert np.array_equal(moments.m[big:big + 64].cpu().numpy(), q.reshape(-1))
    assert not moments.m[:64].any() and not moments.m[big - 64:big].any()


def test_refusals():
    p, g = tensors([100, 200]), tensors([100, 200], seed=1)
    moments = mxq.adamw_moments(p)
    for bad, what in ((dict(params=p[:1]), "length"), (dict(grads=[g[0], g[1].half()]), "float32"), (dict(grads=[g[0], g[1][:100]]), "shape"),
                      (dict(params=[p[0], p[0]], grads=[g[0], g[0]]), "m must be"), (dict(grads=[g[0], g[1].cpu()]), "device"),
                      (dict(moments=mxq.adamw_moments(p[:1])), "m must be"), (dict(step=0), "step"), (dict(seed=-1), "seed"),
                      (dict(copies=[None]), "length"), (dict(copies=[p[0], None]), "copies"),
                      (dict(grad_scale=torch.ones(1, device="cuda")), "grad_scale"), (dict(lr=torch.ones((), device="cuda").double()), "lr"),
                      (dict(params=[p[0], torch.randn(20, 20, device="cuda").t()[:10]], grads=[g[0], g[1].view(10, 20)]), "contiguous")):
        args = dict(params=p, grads=g, moments=moments, step=1, **HOW)
        with pytest.raises(ValueError, match=what):
            mxq.adamw_step(**{**args, **bad})
    same = tensors([128, 128])
    with pytest.raises(ValueError, match="different"):
        mxq.adamw_step([same[0], same[0]], same, mxq.adamw_moments(same), 1, **HOW)
    over = torch.randn(300, device="cuda")
    for params, grads in (([over[:200], over[100:]], g[1:] * 2), ([over[:200]], [over[100:]]), ([over[:200]], [over[:200]])):
        with pytest.raises(mxq.MxqError) as e:
            mxq.adamw_step(params, grads, mxq.adamw_moments(params), 1, **HOW)
        assert e.value.code == mxq.EOVERLAP
    for bad in (dict(betas=(1.0, 0.9)), dict(betas=(0.9, -0.1)), dict(eps=-1.0), dict(weight_decay=math.inf), dict(lr=math.nan)):
        with pytest.raises(mxq.MxqError) as e:
            mxq.adamw_step(p, g, moments, 1, **{**HOW, **bad})
        assert e.value.code == mxq.EBADSHAPE
    with pytest.raises(TypeError):
        mxq.adamw_step(p, g, moments, 1.0, **HOW)
