"""The experts' products, grouped routing and AdamW in a run, as a training step uses them.

Two products an expert with a gelu, biases and a residual; the gradients against 64-bit
autograd of the same layer on the values that the casts hold, the choice of experts fixed.
What is left between the two is the casts of the inner values (the activations' and the
gradients'): E4M3 rounds by at most 2^-4 of a value, 2^-4 / sqrt(3) = 3.6% in the norm, and
each gradient goes through one such rounding of either operand and of the hidden values'
gradient, 3 in all where they do not cancel: 11%, and bf16's 0.2% three times.
"""
import pytest
import torch

import mx_block_quantization_gb300 as mxq
from tests.gpu_util import require_gpu
from tests.test_gpu_moe_linear import act64, normal, values

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    yield
    torch.cuda.empty_cache()
    assert mxq.device_status(clear=True) == 0


class Layer:
    """Tokens [T, D] to `experts` pairs of matrices [H, D] and [D, H], k of them each."""

    def __init__(self, T, D, H, E, k, groups, best, seed=0):
        self.T, self.D, self.H, self.E, self.k = T, D, H, E, k
        self.how = dict(groups=groups, best_groups=best, scores="sigmoid", scale=1.5)
        self.x = normal((T, D), seed, dtype=BF16)
        self.router = normal((E, D), seed + 1, D**-0.5)
        self.balance = normal((E,), seed + 2, 0.05)
        self.up, self.down = normal((E, H, D), seed + 3, D**-0.5, BF16), normal((E, D, H), seed + 4, H**-0.5, BF16)
        self.up_bias, self.down_bias = normal((E, H), seed + 5, 0.3), normal((E, D), seed + 6, 0.3)

    def cast(self, w):
        E, n, k = w.shape
        return mxq.quantize_2d_dual(w.view(E * n, k), torch.arange(1, E + 1, dtype=torch.int32, device="cuda") * n)

    def forward(self):
        E, D, H = self.E, self.D, self.H
        self.logits = self.x.float() @ self.router.t()
        self.r = mxq.moe_route_groups(self.logits, self.k, bias=self.balance, **self.how)
        self.plan = mxq.moe_plan(self.r.ids, E)
        offs = self.plan.offs
        self.cx = mxq.quantize_2d_dual(mxq.moe_dispatch(self.x, self.plan), offs)
        self.cu, self.cd = self.cast(self.up), self.cast(self.down)
        h, self.z = mxq.moe_linear(self.cx.q_row, self.cx.s_row, self.cu.q_row.view(E, H, D), self.cu.s_row, offs, bias=self.up_bias,
                                   activation="gelu", preactivation=True)
        self.ch = mxq.quantize_2d_dual(h, offs)
        self.rows = mxq.moe_linear(self.ch.q_row, self.ch.s_row, self.cd.q_row.view(E, D, H), self.cd.s_row, offs, bias=self.down_bias,
                                   residual=mxq.moe_dispatch(self.x, self.plan))
        return mxq.moe_combine(self.rows, self.plan, self.r.weights), self.r.loss

    def backward(self, dy, dloss):
        E, D, H, offs = self.E, self.D, self.H, self.plan.offs
        drows, dweights = mxq.moe_combine_backward(dy, self.rows, self.plan, self.r.weights)
        _, d_down_bias = mxq.moe_linear_backward(drows, offs=offs)
        c = mxq.quantize_2d_dual(drows, offs)
        dh = mxq.moe_linear(c.q_row, c.s_row, self.cd.q_col.view(H, E, D).transpose(0, 1), self.cd.s_col, offs)
        d_down = mxq.moe_weight_gradient(c.q_col, c.s_col, self.ch.q_col, self.ch.s_col, offs)
        dz, d_up_bias = mxq.moe_linear_backward(dh, self.z, offs, activation="gelu")
        c = mxq.quantize_2d_dual(dz, offs)
        dx_rows = mxq.moe_linear(c.q_row, c.s_row, self.cu.q_col.view(D, E, H).transpose(0, 1), self.cu.s_col, offs, residual=drows)
        d_up = mxq.moe_weight_gradient(c.q_col, c.s_col, self.cx.q_col, self.cx.s_col, offs)
        dlogits = mxq.moe_route_groups_backward(self.logits, self.r, dweights, dloss, scores="sigmoid", scale=1.5)
        return dict(up=d_up, down=d_down, up_bias=d_up_bias, down_bias=d_down_bias, logits=dlogits, x=mxq.moe_combine(dx_rows, self.plan))


def wanted(layer, dy, dloss):
    """Output, loss and gradients by autograd in 64 bits from the casts' values of the inputs and weights."""
    E, D, H, T, k = layer.E, layer.D, layer.H, layer.T, layer.k
    leaf = lambda t: t.double().requires_grad_()  # noqa: E731
    up = leaf(values(layer.cu.q_row, layer.cu.s_row).view(E, H, D))
    down = leaf(values(layer.cd.q_row, layer.cd.s_row).view(E, D, H))
    up_bias, down_bias, logits, x = leaf(layer.up_bias), leaf(layer.down_bias), leaf(layer.logits), leaf(layer.x)
    ids = layer.r.ids.long()
    s = torch.sigmoid(logits)
    picked = s.gather(1, ids)
    w = 1.5 * picked / picked.sum(1, keepdim=True)
    y = torch.zeros(T, D, dtype=torch.float64, device="cuda")
    for j in range(k):
        for e in range(E):
            at = (ids[:, j] == e).nonzero()[:, 0]
            h = act64(x[at] @ up[e].t() + up_bias[e], "gelu")
            y = y.index_add(0, at, w[at, j, None] * (h @ down[e].t() + down_bias[e] + x[at]))
    counts = torch.bincount(ids.view(-1), minlength=E).double()
    loss = E / (k * T * T) * (counts * (s / s.sum(1, keepdim=True)).sum(0)).sum()
    ((y * dy.double()).sum() + dloss * loss).backward()
    return y.detach(), loss.detach(), dict(up=up.grad, down=down.grad, up_bias=up_bias.grad, down_bias=down_bias.grad, logits=logits.grad, x=x.grad)


def off(a, b):
    return float((a.double() - b).norm() / b.norm())


@pytest.mark.parametrize("T,D,H,E,k,groups,best", [(700, 128, 256, 8, 2, 4, 2), (1, 256, 128, 4, 1, 1, 1), (300, 384, 128, 24, 3, 8, 3)])
def test_gradients_of_a_layer(T, D, H, E, k, groups, best):
    layer = Layer(T, D, H, E, k, groups, best)
    dy = normal((T, D), 9, dtype=BF16)
    y, loss = layer.forward()
    got = layer.backward(dy, torch.tensor(2.0, device="cuda"))
    want_y, want_loss, want = wanted(layer, dy, 2.0)
    assert float(loss) == pytest.approx(float(want_loss), rel=1e-5)
    assert off(y, want_y) < 0.08            # two roundings: of x and of the hidden values
    for name in want:
        # the bias of the second product has no cast before it; others have up to three
        assert off(got[name], want[name]) < (0.01 if name == "down_bias" else 0.12), name


def test_a_step_captured_and_replayed():
    """Forward, backward and update of all weights in one graph, the step counted on the device."""
    def run(replay):
        layer = Layer(400, 128, 256, 8, 2, 4, 2)
        dy, dloss = normal((400, 128), 9, dtype=BF16), torch.tensor(0.5, device="cuda")
        params = [layer.up, layer.down, layer.up_bias, layer.down_bias]
        moments, t = mxq.adamw_moments(params, 8), torch.ones((), dtype=torch.int64, device="cuda")

        def step():
            y, loss = layer.forward()
            g = layer.backward(dy, dloss)
            mxq.adamw_step(params, [g["up"], g["down"], g["up_bias"], g["down_bias"]], moments, t, lr=1e-3, seed=7)
            t.add_(1)
            return y, loss
        if not replay:
            for _ in range(3):
                out = step()
        else:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                out = step()
            for _ in range(3):
                graph.replay()
        torch.cuda.synchronize()
        return [x.clone() for x in (*params, *out, moments.m, moments.v, moments.m_scale, moments.v_scale)]

    run(False)
    for a, b in zip(run(False), run(True)):
        assert torch.equal(a, b)


def test_two_streams_at_once():
    """Products and steps of two layers on two streams: each as alone."""
    layers = [Layer(500, 256, 384, 8, 2, 4, 2, seed=s) for s in (0, 50)]
    alone = [layer.forward()[0].clone() for layer in layers]
    streams = [torch.cuda.Stream() for _ in layers]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        both = []
        for layer, s in zip(layers, streams):
            with torch.cuda.stream(s):
                both.append(layer.forward()[0])
        torch.cuda.synchronize()
        for a, b in zip(alone, both):
            assert torch.equal(a, b)


def test_refusals_of_the_calls():
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")  # noqa: E731
    q, s, w, sw = u8(256, 128), u8(1024), u8(2, 128, 128), u8(1024)
    offs, x = torch.tensor([128, 256], dtype=torch.int32, device="cuda"), torch.zeros(256, 128, device="cuda")
    for call, what in ((lambda: mxq.moe_linear(q, s, w[0], sw, offs), "3-D"), (lambda: mxq.moe_linear(q, s, w, sw), "2-D"),
                       (lambda: mxq.moe_linear(q, s, w[:1], sw, offs), "2 matrices"), (lambda: mxq.moe_linear(q, s[1:], w, sw, offs), "1024 scales"),
                       (lambda: mxq.moe_linear(q, s, w, sw[:512], offs), "1024 scales"), (lambda: mxq.moe_linear(q, s, w[..., :64], sw, offs), "w must be"),
                       (lambda: mxq.moe_linear(q.float(), s, w, sw, offs), "E4M3"), (lambda: mxq.moe_linear(q, s, w, sw, offs.long()), "offs"),
                       (lambda: mxq.moe_linear(q, s, w, sw, offs, activation="tanh"), "activation"),
                       (lambda: mxq.moe_linear(q, s, w, sw, offs, bias=x[0]), "bias"), (lambda: mxq.moe_linear(q, s, w, sw, offs, residual=x), "residual"),
                       (lambda: mxq.moe_linear(q, s, w, sw, offs, dtype=torch.float16), "dtype"),
                       (lambda: mxq.moe_linear(q, s, w, sw, offs, out=x[:128]), "out must be"),
                       (lambda: mxq.moe_linear(q, s, w, sw, offs, out=x.t().contiguous().t()), "unit column"),
                       (lambda: mxq.moe_linear_backward(x, None, offs, activation="relu"), "z is needed"),
                       (lambda: mxq.moe_linear_backward(x, x.bfloat16(), offs, activation="relu"), "type"),
                       (lambda: mxq.moe_weight_gradient(q.t().contiguous(), s, q.t().contiguous(), s, offs, accumulate=True), "accumulate"),
                       (lambda: mxq.moe_weight_gradient(q.t().contiguous(), s, u8(128, 128), s, offs), "b must be"),
                       (lambda: mxq.moe_route_groups(x, 2, scores="relu"), "scores"), (lambda: mxq.moe_route_groups(x, 2, bias=x[0, :5]), "bias")):
        with pytest.raises(ValueError, match=what):
            call()
    for call in (lambda: mxq.moe_linear(q[:100], s[:400], w, sw, offs), lambda: mxq.moe_linear(q, s, w.expand(2, 128, 128)[:1].expand(2, 128, 128), sw, offs),
                 lambda: mxq.moe_route_groups(x, 2, groups=3), lambda: mxq.moe_route_groups(x, 0), lambda: mxq.moe_route_groups(x, -1),
                 lambda: mxq.moe_route_groups(x, 9, groups=16), lambda: mxq.moe_route_groups(x, (1 << 32) + 2)):
        with pytest.raises(mxq.MxqError) as e:
            call()
        assert e.value.code == mxq.EBADSHAPE
    for call in (lambda: mxq.moe_linear_backward(x, x, offs, activation="relu", out=(torch.zeros_like(x), x[:2])),
                 lambda: mxq.moe_linear(q, s, w, sw, offs, out=x, bias=x[:2])):
        with pytest.raises(mxq.MxqError) as e:
            call()
        assert e.value.code == mxq.EOVERLAP
