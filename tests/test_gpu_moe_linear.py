"""The experts' products on the cast's bytes against the same products in 64 bits.

Tolerances: a product of two E4M3 values has 8 bits and is exact; each step of 32 along
K rounds its sum of products and the addition to the accumulator, taken as two
truncations in fp32, 2^-23 of the sum S of all products' sizes each.  An activation
stretches that by at most 1.13 (the largest slope, of gelu) and adds 2^-20 of its value
(the hardware's exponential and reciprocal, 2^-22 each, and three fp32 operations); the
bias and the residual add a rounding of 2^-24 of what they meet, and the result's type
half a step.
"""
import pytest
import torch

import mx_block_quantization_gb300 as mxq
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    yield
    torch.cuda.empty_cache()
    assert mxq.device_status(clear=True) == 0


def normal(shape, seed, scale=1.0, dtype=F32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def values(q, s):
    """E4M3 bytes [R, C] with blocked E8M0 scales, in 64 bits."""
    r, c = q.shape
    scale = s.reshape(r // 128, c // 128, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(r, c // 32).double() - 127
    v = q.contiguous().view(torch.float8_e4m3fn).double() * torch.exp2(scale).repeat_interleave(32, 1)
    return v


def ends_of(blocks):
    return torch.tensor([128 * b for b in blocks], dtype=torch.int32).cumsum(0).int()


def act64(z, name):
    if name == "relu":
        return torch.relu(z)
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return 0.5 * z * (1 + torch.tanh((2 / torch.pi) ** 0.5 * (z + 0.044715 * z**3)))
    return z


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


class Problem:
    """Rows in groups of `blocks` 128-row blocks, and `tail` blocks behind the last."""

    def __init__(self, blocks, tail, N, K, seed=0, dtype=BF16, dense=False):
        self.blocks, self.N, self.K, self.dtype = blocks, N, K, dtype
        self.G, self.M = len(blocks), 128 * (sum(blocks) + tail)
        self.offs = None if dense else ends_of(blocks).cuda()
        x = normal((self.M, K), seed, dtype=BF16) * torch.exp(normal((K,), seed + 1)).to(BF16)
        w = normal((self.G * N, K), seed + 2, K**-0.5, BF16)
        cx, cw = mxq.quantize_2d_dual(x, self.offs), mxq.quantize_2d_dual(w)
        self.q, self.s, self.w, self.sw = cx.q_row, cx.s_row, cw.q_row.view(self.G, N, K), cw.s_row
        self.bias = normal((self.G, N), seed + 3)
        self.residual = normal((self.M, N), seed + 4, dtype=dtype)

    def wanted(self, bias=None):
        """z, and the sum of the products' sizes."""
        z = torch.zeros(self.M, self.N, dtype=torch.float64, device="cuda")
        size = torch.zeros_like(z)
        x, lo, per = values(self.q, self.s), 0, self.N * self.K // 32
        for e, b in enumerate(self.blocks):
            hi = lo + 128 * b
            w = values(self.w[e], self.sw[e * per:(e + 1) * per])
            z[lo:hi] = x[lo:hi] @ w.t()
            size[lo:hi] = x[lo:hi].abs() @ w.abs().t()
            if bias is not None:
                z[lo:hi] += bias[e].double()
            lo = hi
        return z, size, lo

    def check(self, activation=None, bias=None, residual=None, keep=False, **how):
        w = self.w if self.offs is not None else self.w[0]
        b = bias if self.offs is not None or bias is None else bias[0]
        got = mxq.moe_linear(self.q, self.s, w, self.sw, self.offs, bias=b, activation=activation, residual=residual,
                             preactivation=keep, dtype=self.dtype, **how)
        y, z = got if keep else (got, None)
        before = None if residual is None else residual.double().clone()
        self.compare(y, z, activation, bias, before)
        return got

    def compare(self, y, z, activation, bias, residual):
        want, size, end = self.wanted(bias)
        off = self.K / 32 * 2 * 2.0**-23 * size + 2.0**-24 * want.abs()
        if z is not None:
            assert z.dtype == self.dtype
            assert bool(((z.double() - want).abs() <= off + half_step(self.dtype) * (want.abs() + off)).all())
            assert not z[end:].any()
        want_y = act64(want, activation)
        off = 1.13 * off + (2.0**-20 * want_y.abs() if activation else 0)
        if residual is not None:
            want_y = want_y + residual
            off = off + 2.0**-24 * want_y.abs()
        assert y.dtype == self.dtype and y.shape == (self.M, self.N)
        err = (y.double() - want_y).abs()[:end]
        assert bool((err <= (off + half_step(self.dtype) * (want_y.abs() + off))[:end]).all()), float(err.max())
        assert not y[end:].any()


@pytest.mark.parametrize("N,K", [(128, 128), (256, 128), (128, 384), (256, 2048), (384, 1152), (640, 256)])
def test_one_group(N, K):
    Problem([1], 0, N, K, dense=True).check()
    Problem([3], 0, N, K, dtype=F32).check()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("blocks,tail", [([1, 2, 3], 0), ([0, 5, 0, 1, 0], 2), ([7, 4, 1, 1, 6, 0, 0, 3], 1), ([17, 2], 0),
                                         ([0, 0, 1], 0), ([1] * 40, 3), ([2] * 33, 0), ([25], 4)])
def test_groups(blocks, tail, dtype):
    Problem(blocks, tail, 384, 512, seed=len(blocks), dtype=dtype).check()


def test_rows_in_no_group():
    p = Problem([0, 0, 0], 3, 256, 256)
    assert not p.check().any()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("activation", [None, "relu", "silu", "gelu"])
@pytest.mark.parametrize("bias,residual,keep", [(True, False, True), (False, True, False), (True, True, True)])
def test_epilogue(activation, bias, residual, keep, dtype):
    p = Problem([3, 0, 2, 4], 1, 640, 768, seed=5, dtype=dtype)
    p.check(activation, p.bias if bias else None, p.residual if residual else None, keep)


def test_many_tiles_a_pair():
    """Tiles of both heights follow one another on a pair, on both accumulators."""
    p = Problem([5, 1, 8, 3, 2, 9, 1, 1, 6, 7, 4, 3, 0, 11, 1, 2], 2, 2176, 640, seed=3)
    first = p.check("silu", p.bias, None, True)
    again = p.check("silu", p.bias, None, True)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_strides_and_places(dtype):
    """Operands, outputs and residual with gaps between their rows, at odd places."""
    p = Problem([2, 3], 1, 384, 256, seed=11, dtype=dtype)
    plain = p.check("gelu", p.bias, p.residual, True)
    room = torch.zeros(p.M, 272, dtype=torch.uint8, device="cuda")
    room[:, :256] = p.q
    p.q = room[:, :256]
    wide = torch.zeros(2, 390, 288, dtype=torch.uint8, device="cuda")
    wide[:, :384, :256] = p.w
    p.w = wide[:, :384, :256]
    outs = [torch.full((p.M, 391), 7.0, dtype=dtype, device="cuda") for _ in range(2)]
    kept = torch.full((p.M, 387), 5.0, dtype=dtype, device="cuda")
    kept[:, 3:] = p.residual
    y, z = mxq.moe_linear(p.q, p.s, p.w, p.sw, p.offs, bias=p.bias.to(BF16).float(), activation="gelu", residual=kept[:, 3:],
                          preactivation=True, out=(outs[0][:, 5:389], outs[1][:, 1:385]))
    p.compare(y, z, "gelu", p.bias.to(BF16).float(), p.residual.double())
    for o, lo in zip(outs, (5, 1)):
        assert bool((o[:, :lo] == 7).all()) and bool((o[:, lo + 384:] == 7).all())
    b16 = mxq.moe_linear(p.q, p.s, p.w, p.sw, p.offs, bias=p.bias.to(BF16), activation="gelu", residual=kept[:, 3:],
                         preactivation=True, dtype=dtype)
    assert torch.equal(b16[0], y) and torch.equal(b16[1], z)
    same = kept[:, 3:]
    assert mxq.moe_linear(p.q, p.s, p.w, p.sw, p.offs, bias=p.bias, activation="gelu", residual=same, out=same) is same
    assert torch.equal(same, plain[0])


def test_a_scale_of_nan_is_nan_where_it_is_used():
    p = Problem([1, 1], 0, 128, 256, seed=2)
    p.s[0] = 255                       # row 0, the first 32 of K
    y = mxq.moe_linear(p.q, p.s, p.w, p.sw, p.offs)
    nan = torch.isnan(y)
    assert bool(nan[0].all()) and not nan[1:].any()


def test_the_rows_gradient_is_the_same_product():
    """dx = dz w with the weights' column-wise bytes, one cast of the whole stack."""
    G, N, K, blocks = 3, 256, 384, [2, 1, 4]
    offs, M = ends_of(blocks).cuda(), 128 * 7
    w = normal((G * N, K), 1, 0.05, BF16)
    per = torch.arange(1, G + 1, dtype=torch.int32, device="cuda") * N
    cw = mxq.quantize_2d_dual(w, per)
    dz = mxq.quantize_2d_dual(normal((M, N), 2, dtype=BF16), offs)
    wt = cw.q_col.view(K, G, N).transpose(0, 1)
    dx = mxq.moe_linear(dz.q_row, dz.s_row, wt, cw.s_col, offs, dtype=F32)
    lo = 0
    for e, b in enumerate(blocks):
        hi = lo + 128 * b
        a = values(dz.q_row[lo:hi], dz.s_row[lo * N // 32:hi * N // 32])
        v = values(wt[e], cw.s_col[e * N * K // 32:(e + 1) * N * K // 32])
        off = N / 32 * 2 * 2.0**-23 * (a.abs() @ v.abs().t())
        want = a @ v.t()
        assert bool(((dx[lo:hi].double() - want).abs() <= off + 2.0**-24 * want.abs()).all())
        lo = hi


def weights_wanted(dz, x, blocks, N, K):
    want = torch.zeros(len(blocks), N, K, dtype=torch.float64, device="cuda")
    size, lo = torch.zeros_like(want), 0
    for e, b in enumerate(blocks):
        hi = lo + 128 * b
        if b:
            a = values(dz.q_col[:, lo:hi], dz.s_col[N * lo // 32:N * hi // 32])
            v = values(x.q_col[:, lo:hi], x.s_col[K * lo // 32:K * hi // 32])
            want[e], size[e] = a @ v.t(), a.abs() @ v.abs().t()
        lo = hi
    return want, size


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("blocks,tail", [([1], 0), ([3, 0, 1, 6], 1), ([0, 0], 2), ([2] * 9, 0), ([9, 1, 0, 0, 14], 0)])
@pytest.mark.parametrize("N,K", [(128, 128), (384, 256), (256, 640), (896, 1152)])
def test_weight_gradient(blocks, tail, N, K, dtype):
    M, offs = 128 * (sum(blocks) + tail), ends_of(blocks).cuda()
    dz, x = (mxq.quantize_2d_dual(normal((M, n), seed, dtype=BF16), offs) for n, seed in ((N, 1), (K, 2)))
    want, size = weights_wanted(dz, x, blocks, N, K)
    off = max(max(blocks), 1) * 4 * 2 * 2.0**-23 * size
    got = mxq.moe_weight_gradient(dz.q_col, dz.s_col, x.q_col, x.s_col, offs, dtype=dtype)
    assert bool(((got.double() - want).abs() <= off + half_step(dtype) * (want.abs() + off)).all())
    # added to what is there, in rows with gaps and matrices further apart
    room = normal((len(blocks), N + 2, K + 3), 3, 20.0, dtype)
    before, out = room.double(), room[:, 1:N + 1, 2:K + 2]
    assert mxq.moe_weight_gradient(dz.q_col, dz.s_col, x.q_col, x.s_col, offs, out=out, accumulate=True) is out
    want = want + before[:, 1:N + 1, 2:K + 2]
    assert bool(((out.double() - want).abs() <= off + (2.0**-24 + half_step(dtype)) * (want.abs() + off)).all())
    room[:, 1:N + 1, 2:K + 2] = 0
    before[:, 1:N + 1, 2:K + 2] = 0
    assert torch.equal(room.double(), before)


def test_weight_gradient_without_offs():
    x, dz = (mxq.quantize_2d_dual(normal((640, n), seed, dtype=BF16)) for n, seed in ((256, 4), (384, 5)))
    want, size = weights_wanted(dz, x, [5], 384, 256)
    got = mxq.moe_weight_gradient(dz.q_col, dz.s_col, x.q_col, x.s_col)
    assert got.shape == (384, 256)
    assert bool(((got.double() - want[0]).abs() <= 20 * 2 * 2.0**-23 * size[0] + 2.0**-24 * want[0].abs()).all())


def test_weight_gradient_of_no_rows():
    none = torch.empty(128, 0, dtype=torch.uint8, device="cuda")
    scales = torch.empty(0, dtype=torch.uint8, device="cuda")
    offs = torch.zeros(3, dtype=torch.int32, device="cuda")
    out = torch.full((3, 128, 128), 3.0, device="cuda")
    mxq.moe_weight_gradient(none, scales, none, scales, offs, out=out, accumulate=True)
    assert bool((out == 3).all())
    mxq.moe_weight_gradient(none, scales, none, scales, offs, out=out)
    assert not out.any()


def slope64(z, name):
    z = z.clone().requires_grad_()
    act64(z, name).sum().backward()
    return z.grad


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("activation", [None, "relu", "silu", "gelu"])
@pytest.mark.parametrize("blocks,tail,N", [([1], 0, 128), ([3, 0, 2], 2, 384), ([20, 1, 0], 0, 2176), ([0], 1, 128)])
def test_epilogue_gradient(blocks, tail, N, activation, dtype):
    """dz is a product of fp32 values that are right to 2^-20, rounded to its type; dbias
    is summed in fp32, each of its at most 2560 additions off by 2^-24 of the sum of sizes."""
    M, offs = 128 * (sum(blocks) + tail), ends_of(blocks).cuda()
    end = 128 * sum(blocks)
    dy, z = normal((M, N), 1, dtype=dtype), normal((M, N), 2, 2.0, dtype)
    want = dy.double() * slope64(z.double(), activation) if activation else dy.double()
    got, dbias = mxq.moe_linear_backward(dy, z, offs, activation=activation)
    if activation:
        assert bool(((got.double() - want).abs()[:end] <= (half_step(dtype) + 2.0**-20) * want.abs()[:end] + 2.0**-20 * dy.double().abs()[:end]).all())
        assert not got[end:].any()
    else:
        assert got is dy
    lo = 0
    for e, b in enumerate(blocks):
        hi = lo + 128 * b
        d = want[lo:hi]
        off = (2.0**-20 + 128 * b * 2.0**-24) * d.abs().sum(0) + 2.0**-20 * dy.double()[lo:hi].abs().sum(0)
        assert bool(((dbias[e].double() - d.sum(0)).abs() <= off).all())
        lo = hi
    # strided, in place, the same bits
    room = torch.full((M, N + 5), 3.0, dtype=dtype, device="cuda")
    room[:, 3:N + 3] = dy
    if activation:
        at = room[:, 3:N + 3]
        again, db = mxq.moe_linear_backward(at, z, offs, activation=activation, out=(at, torch.empty_like(dbias)))
        assert torch.equal(again, got) and bool((room[:, :3] == 3).all()) and bool((room[:, N + 3:] == 3).all())
        one, db1 = mxq.moe_linear_backward(dy, z, None, activation=activation)
        assert torch.equal(one[:end], got[:end]) and db1.shape == (N,)


def test_slopes_at_the_ends():
    z = torch.tensor([-torch.inf, -100.0, -0.0, 0.0, 100.0, torch.inf, torch.nan] + [1.0] * 121, device="cuda").expand(128, 128).contiguous()
    dy = torch.ones_like(z)
    for name, want in (("relu", [0, 0, 0, 0, 1, 1]), ("silu", [None, 0, 0.5, 0.5, 1, None]), ("gelu", [None, 0, 0.5, 0.5, 1, None])):
        dz = mxq.moe_linear_backward(dy, z, activation=name)[0][0]
        for got, v in zip(dz.tolist(), want):
            assert v is None or abs(got - v) < 1e-6
        assert torch.isnan(dz[6])


@pytest.mark.parametrize("name", ["silu", "gelu"])
def test_slopes_of_large_values(name):
    """1 above and 0 below, up to infinity: no power of z overflows on the way."""
    sizes = [60.0, 70.0, 127.0, 130.0, 1e6, 1e12, 2e13, 1e19, 2e19, 1e30, 3e38, torch.inf]
    for dtype in (F32, BF16):
        z = torch.tensor(sizes + [1.0] * (128 - len(sizes)), device="cuda").to(dtype).expand(128, 128).contiguous()
        for sign in (1, -1):
            dz = mxq.moe_linear_backward(torch.ones_like(z), sign * z, activation=name)[0][:, :len(sizes)]
            assert bool(((dz - (1 if sign > 0 else 0)).abs() <= 1e-20).all())


@pytest.mark.parametrize("bad", [[128, 64, 256], [64, 128, 256], [-128, 128, 256], [128, 256, 640], [256, 128, 384]])
def test_offs_that_are_no_ends_write_nothing(bad):
    p = Problem([1, 1, 2], 0, 128, 128)
    offs = torch.tensor(bad, dtype=torch.int32, device="cuda")
    c = mxq.quantize_2d_dual(normal((512, 128), 1, dtype=BF16))
    y, z = (torch.full((512, 128), 7.0, dtype=BF16, device="cuda") for _ in range(2))
    dw, db = torch.full((3, 128, 128), 7.0, device="cuda"), torch.full((3, 128), 7.0, device="cuda")
    for call in (lambda: mxq.moe_linear(p.q, p.s, p.w, p.sw, offs, preactivation=True, out=(y, z)),
                 lambda: mxq.moe_weight_gradient(c.q_col, c.s_col, c.q_col, c.s_col, offs, out=dw),
                 lambda: mxq.moe_linear_backward(p.residual, p.residual, offs, activation="silu", out=(y, db))):
        call()
        assert mxq.device_status(clear=True) == mxq.DEV_BADOFFS
        for t in (y, z, dw, db):
            assert bool((t == 7).all())


def test_captured_and_replayed_with_other_groups():
    """offs are read on the device: a captured call follows them."""
    p = Problem([2, 3, 1], 2, 256, 384, seed=8)
    p.check("silu", p.bias, None)
    y = torch.empty(p.M, p.N, dtype=BF16, device="cuda")
    call = lambda: mxq.moe_linear(p.q, p.s, p.w, p.sw, p.offs, bias=p.bias, activation="silu", out=y)  # noqa: E731
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for blocks in ([2, 3, 1], [0, 8, 0], [1, 1, 1], [4, 0, 4]):
        p.blocks = blocks
        p.offs.copy_(ends_of(blocks))
        graph.replay()
        torch.cuda.synchronize()
        p.compare(y, None, "silu", p.bias, None)


def test_streams_and_no_rows():
    p = Problem([1, 2], 0, 256, 256, seed=4)
    want = mxq.moe_linear(p.q, p.s, p.w, p.sw, p.offs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = mxq.moe_linear(p.q, p.s, p.w, p.sw, p.offs, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    none = mxq.moe_linear(p.q[:0], p.s[:0], p.w, p.sw, torch.zeros(2, dtype=torch.int32, device="cuda"))
    assert none.shape == (0, 256)
    dz, db = mxq.moe_linear_backward(want[:0], want[:0], torch.zeros(2, dtype=torch.int32, device="cuda"), activation="relu")
    assert dz.shape == (0, 256) and db.shape == (2, 256) and not db.any()
