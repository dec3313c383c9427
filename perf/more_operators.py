"""More training operators around the MXFP8 cast, as cases to measure and compare.

Three operators of a mixture-of-experts training step, each in its plain form
(elementary torch operations in 32 bits, rounded once at the end) and through
the package's own calls:

* linear   the experts' products on the cast's bytes: rows in 128-row groups times
           each group's weights, with bias, activation and residual; the gradient
           of the activation and the bias; and the weights' gradient per group.
* route    router logits -> scores (sigmoid or softmax), a bias that balances the
           choice, groups of experts, the k experts of each token among the best
           groups, their weights and the balance loss; then the logits' gradient.
* adamw    a step over many tensors at once, with moments in 32 bits or in MXFP8.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
BETAS = (0.9, 0.95)
EPS = 1e-8
DECAY = 0.1
LR = 1e-3


# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one small dense layer on one block of rows: latency of a call
        {"name": "linear small", "op": "linear", "way": "forward", "experts": 0, "rows": 128, "inner": 512,
         "outer": 256, "activation": "silu", "bias": True, "residual": False, "keep": False, "type": "bf16"},
        # a decoding step: 128 routed rows over 64 experts, the time is reading their weights
        {"name": "linear decode", "op": "linear", "way": "forward", "experts": 64, "rows": 128, "inner": 7168,
         "outer": 2048, "activation": "none", "bias": False, "residual": False, "keep": False, "type": "bf16"},
        # the up projection of the grouped cast's workload: 57344 routed rows of width 7168 in 64
        # uneven groups, with what backward needs
        {"name": "linear experts", "op": "linear", "way": "forward", "experts": 64, "rows": 57344, "inner": 7168,
         "outer": 2048, "activation": "gelu", "bias": True, "residual": False, "keep": True, "type": "bf16"},
        # a shared expert: every token through one large matrix, onto the residual stream
        {"name": "linear dense", "op": "linear", "way": "forward", "experts": 0, "rows": 16384, "inner": 4096,
         "outer": 8192, "activation": "none", "bias": False, "residual": True, "keep": False, "type": "f32"},
        # the weights' gradient of narrower experts, added to what earlier micro-batches left
        {"name": "linear weights", "op": "linear", "way": "weights", "experts": 24, "rows": 40009, "inner": 2176,
         "outer": 1408, "activation": "none", "bias": False, "residual": True, "keep": False, "type": "f32"},
        # gradient of activation and bias over the grouped rows: memory traffic
        {"name": "linear epilogue", "op": "linear", "way": "epilogue", "experts": 64, "rows": 57344, "inner": 128,
         "outer": 4096, "activation": "silu", "bias": True, "residual": False, "keep": True, "type": "bf16"},
        # a micro-batch of a few tokens: latency of the two calls
        {"name": "route small", "op": "route", "tokens": 32, "experts": 64, "groups": 8, "best": 4, "k": 6,
         "scores": "sigmoid", "renorm": True, "type": "f32", "masked": 0.0, "pad": 0},
        # a long packed batch with padding tokens over 256 experts in 8 groups
        {"name": "route long", "op": "route", "tokens": 131071, "experts": 256, "groups": 8, "best": 4, "k": 8,
         "scores": "sigmoid", "renorm": True, "type": "f32", "masked": 0.1, "pad": 0},
        # softmax scores, bf16 logits with many equal ones, an odd number of tokens, strided rows
        {"name": "route softmax", "op": "route", "tokens": 10007, "experts": 150, "groups": 5, "best": 3, "k": 6,
         "scores": "softmax", "renorm": False, "type": "bf16", "masked": 0.0, "pad": 3},
        # norms, biases and a router: small tensors, latency
        {"name": "adamw small", "op": "adamw", "tensors": 9, "least": 64, "most": 20000, "bits": 32,
         "type": "f32", "gradient": "f32", "copies": False},
        # fp32 weights with bf16 copies for the cast, gradients in bf16
        {"name": "adamw layers", "op": "adamw", "tensors": 48, "least": 4096, "most": 50000000, "bits": 32,
         "type": "f32", "gradient": "bf16", "copies": True},
        # the same with moments in MXFP8
        {"name": "adamw eight bits", "op": "adamw", "tensors": 48, "least": 4096, "most": 50000000, "bits": 8,
         "type": "f32", "gradient": "bf16", "copies": True},
    ]


def draw(rng):
    def log(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["linear", "linear", "route", "adamw"])
    kind = rng.choice(["f32", "bf16"])
    if op == "linear":
        way = rng.choice(["forward", "forward", "weights", "epilogue"])
        inner, outer = 128 * log(1, 64), 128 * log(1, 64)
        # no more weights, products (padded groups included) and elements than the listed cases
        experts = rng.choice([0, log(1, 96), log(1, 96)])
        experts = min(experts, 64 * 2048 * 7168 // (inner * outer))
        most = min(65536, 16384 * 4096 * 8192 // (inner * outer) if way != "epilogue" else 57344 * 4096 // outer)
        rows = log(1, max(1, most - 128 * experts))
        if experts == 0:
            rows = max(128, rows // 128 * 128)
        gradient = way != "forward"
        return {"op": op, "way": way, "experts": experts, "rows": rows, "inner": inner, "outer": outer,
                "activation": rng.choice(["none", "relu", "gelu", "silu"]) if way != "weights" else "none",
                "bias": way == "epilogue" or (not gradient and rng.random() < 0.5),
                "residual": way != "epilogue" and rng.random() < 0.5,
                "keep": way == "epilogue" or (not gradient and rng.random() < 0.5), "type": kind}
    if op == "route":
        groups, size = log(1, 16), log(2, 64)
        best = rng.randint(1, groups)
        experts = groups * size
        return {"op": op, "tokens": min(log(1, 131071), 131071 * 256 // experts), "experts": experts, "groups": groups,
                "best": best, "k": rng.randint(1, min(8, best * size)), "scores": rng.choice(["sigmoid", "softmax"]),
                "renorm": rng.random() < 0.5, "type": kind, "masked": rng.choice([0.0, 0.1, 0.5]),
                "pad": rng.choice([0, 0, 1, 8])}
    tensors, most = log(1, 150), log(64, 50000000)
    most = min(most, 48 * 50000000 // tensors // 8)
    return {"op": op, "tensors": tensors, "least": log(1, min(most, 4096)), "most": most, "bits": rng.choice([32, 8]),
            "type": kind, "gradient": rng.choice(["f32", "bf16"]), "copies": kind == "f32" and rng.random() < 0.5}


def _rows_padded(case):
    """Rows that hold the routed ones in groups of whole 128 rows, whichever way they are routed."""
    if not case["experts"]:
        return case["rows"]
    return (case["rows"] + 127 * min(case["experts"], case["rows"])) // 128 * 128


def _sizes(case):
    """Elements of each tensor, spread over the logarithm of the range, odd ones among them."""
    n, lo, hi = case["tensors"], case["least"], case["most"]
    at = [((7 * i + 3) % n) / max(1, n - 1) for i in range(n)]
    return [max(1, int(round(lo * (hi / lo) ** a))) for a in at]


def _starts(sizes):
    """Where each tensor's moments begin, each at a multiple of 128, and where the last end."""
    starts, at = [], 0
    for n in sizes:
        starts.append(at)
        at += (n + 127) // 128 * 128
    return starts, at


def work(case):
    c = case
    if c["op"] == "adamw":
        n = sum(_sizes(c))
        p, g = (4 if c["type"] == "f32" else 2), (4 if c["gradient"] == "f32" else 2)
        m = 16 if c["bits"] == 32 else 4 + 4 / 32
        return {"bytes": n * (2 * p + g + m + (2 if c["copies"] else 0)), "flops": 15 * n}
    e = 4 if c["type"] == "f32" else 2
    if c["op"] == "route":
        n, s = c["tokens"] * c["experts"], c["tokens"] * c["k"]
        # logits in, their gradient out; weights and ids out, the weights' gradient in
        return {"bytes": 2 * n * e + s * 12 + c["experts"] * 8, "flops": 25 * n}
    # the rows of a group's last 128 count: they are part of the layout that the cast gives
    x, k, n = c["experts"] or 1, c["inner"], c["outer"]
    routed = c["rows"] + (64 * min(x, c["rows"]) if c["experts"] else 0)
    used = min(x, c["rows"])
    operand = 1 + 1 / 32
    if c["way"] == "forward":
        outs = 1 + (1 if c["keep"] else 0) + (1 if c["residual"] else 0)
        return {"bytes": operand * (routed * k + used * k * n) + outs * e * routed * n + (4 * x * n if c["bias"] else 0),
                "flops": 2 * routed * k * n}
    if c["way"] == "weights":
        return {"bytes": operand * routed * (k + n) + e * x * k * n * (2 if c["residual"] else 1), "flops": 2 * routed * k * n}
    return {"bytes": e * routed * n * (3 if c["activation"] != "none" else 1) + 4 * x * n, "flops": 12 * routed * n}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _blocked(s):
    """A scale matrix [R, C] in the 128x4 blocked layout."""
    r, c = s.shape
    return s.view(r // 128, 4, 32, c // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _cast(x):
    """E4M3 bytes and E8M0 scale bytes [.., C/32] of x in 1x32 blocks: the smallest power
    of two that brings the largest value of a block within 448."""
    rows, cols = x.shape
    blocks = x.float().view(rows, cols // 32, 32)
    bits = blocks.abs().amax(2).view(torch.int32)
    scale = ((bits >> 23) - 8 + ((bits & 0x7FFFFF) > 0x600000).int()).clamp(min=0)
    up = ((254 - scale) << 23).view(torch.float32)
    q = (blocks * up[..., None]).to(torch.float8_e4m3fn).view(torch.uint8).view(rows, cols)
    return q, scale.to(torch.uint8)


def _by_groups(s, ends, rows):
    """Scales [N, M/32] along the grouped rows: one blocked slab for each group, zeros behind the last."""
    slabs = [_blocked(s[:, lo // 32:hi // 32].contiguous()) for lo, hi in zip([0] + ends[:-1], ends) if hi > lo]
    slabs.append(torch.zeros(s.shape[0] * (rows - ends[-1]) // 32, dtype=torch.uint8, device=s.device))
    return torch.cat(slabs)


def _grouping(case, g):
    """Ends of the groups (a list and the tensor that the cast takes), and which rows hold a routed one."""
    rows, e = _rows_padded(case), case["experts"]
    if not e:
        return [rows], None, torch.ones(rows, dtype=torch.bool, device="cuda")
    liked = torch.randn(e, generator=g, device="cuda") * 0.5
    ids = (torch.rand(case["rows"], e, generator=g, device="cuda").log().neg().log().neg() + liked).argmax(1)
    counts = torch.bincount(ids, minlength=e)
    ends = torch.cumsum((counts + 127) // 128 * 128, 0)
    at = torch.arange(rows, device="cuda")
    group = torch.searchsorted(ends, at, right=True).clamp(max=e - 1)
    live = at < ends[-1]
    live &= at - (ends - (counts + 127) // 128 * 128)[group] < counts[group]
    return ends.tolist(), ends.int(), live


def _normal(shape, g, kind="f32", scale=1.0, pad=0):
    """Normal values; with `pad`, rows that lie further apart than they are long."""
    *lead, n = shape
    x = torch.randn(*lead, n + pad, generator=g, device="cuda") * scale
    return x.to(TYPES[kind])[..., :n]


def _linear_inputs(c, g):
    ends, offs, live = _grouping(c, g)
    rows, e, k, n = _rows_padded(c), c["experts"] or 1, c["inner"], c["outer"]
    s = {"case": c, "ends": ends, "offs": offs}
    if c["way"] == "epilogue":
        s["dy"] = _normal((rows, n), g, c["type"], 0.02) * live[:, None].to(TYPES[c["type"]])
        s["z"] = _normal((rows, n), g, c["type"], 1.5)
        return s
    # activations with a few strong channels; padding rows are zero
    x = _normal((rows, k), g) * torch.exp(0.5 * torch.randn(k, generator=g, device="cuda")) * live[:, None]
    if c["way"] == "weights":
        dz = _normal((rows, n), g, scale=0.02) * live[:, None]
        for name, t in (("x", x), ("dz", dz)):
            q, scale = _cast(t.t().contiguous())
            s[name + "_q"], s[name + "_s"] = q, _by_groups(scale, ends, rows)
        s["sum"] = _normal((e, n, k), g, c["type"], 0.1) if c["residual"] else None
        return s
    q, scale = _cast(x)
    s["x_q"], s["x_s"] = q, _blocked(scale)
    q, scale = _cast(_normal((e * n, k), g, scale=1 / math.sqrt(k)))
    s["w_q"], s["w_s"] = q.view(e, n, k), _blocked(scale)
    s["bias"] = _normal((e, n), g, scale=0.2) if c["bias"] else None
    s["residual"] = _normal((rows, n), g, c["type"]) if c["residual"] else None
    return s


def _moments(c, sizes, g):
    """Moments as a training run leaves them, and their bytes for moments in MXFP8."""
    total = _starts(sizes)[1]
    inside = torch.zeros(total, dtype=torch.bool, device="cuda")
    for n, at in zip(sizes, _starts(sizes)[0]):
        inside[at:at + n] = True
    spread = torch.exp(torch.randn(total, generator=g, device="cuda")) * 1e-2
    m = torch.randn(total, generator=g, device="cuda") * spread * 0.3 * inside
    r = spread * (0.5 + torch.rand(total, generator=g, device="cuda")) * inside
    if c["bits"] == 32:
        return m, r * r, None, None
    (mq, ms), (vq, vs) = _cast(m.view(1, -1)), _cast(r.view(1, -1))
    return mq.view(-1), vq.view(-1), ms.view(-1), vs.view(-1)


def prepare(case, seed):
    c, g = case, torch.Generator(device="cuda").manual_seed(seed)
    if c["op"] == "linear":
        return _linear_inputs(c, g)
    if c["op"] == "route":
        t, e = c["tokens"], c["experts"]
        liked = torch.randn(e, generator=g, device="cuda")
        logits = torch.randn(t, e + c["pad"], generator=g, device="cuda") * 1.5
        logits[:, :e] += liked
        mask = None
        if c["masked"]:
            mask = torch.rand(t, generator=g, device="cuda") >= c["masked"]
            mask[0] = True
        # a bias that has grown against the experts that are liked
        bias = -0.05 * liked + 0.01 * torch.randn(e, generator=g, device="cuda")
        return {"case": c, "logits": logits.to(TYPES[c["type"]])[:, :e], "mask": mask, "bias": bias, "scale": 2.5,
                "dweights": torch.randn(t, c["k"], generator=g, device="cuda") * 0.1,
                "dloss": torch.rand((), generator=g, device="cuda") * 0.01 + 0.005}
    sizes = _sizes(c)
    starts, total = _starts(sizes)
    params = (torch.randn(total, generator=g, device="cuda") * 0.02).to(TYPES[c["type"]])
    grads = (torch.randn(total, generator=g, device="cuda") * 1e-2).to(TYPES[c["gradient"]])
    copies = params.to(torch.bfloat16) if c["copies"] else None
    cut = lambda t: [t[at:at + n] for n, at in zip(sizes, starts)]  # noqa: E731
    return {"case": c, "all_params": params, "params": cut(params), "grads": cut(grads), "all_copies": copies,
            "copies": cut(copies) if c["copies"] else None, "moments": _moments(c, sizes, g), "seed": seed, "step": 10,
            "grad_scale": torch.rand((), generator=g, device="cuda") * 0.5 + 0.5, "starts": starts}


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _scales(s):
    """2^(byte - 127), exact."""
    return torch.where(s > 0, (s.int() << 23).view(torch.float32), 2.0**-127)


def _unblocked(s, rows, cols):
    return s.view(rows // 128, cols // 4, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rows, cols)


def _decode(q, s):
    """Values of E4M3 bytes [R, C] with scale bytes [R, C/32]; 4 significant bits each."""
    r, n = q.shape
    return (q.view(torch.float8_e4m3fn).float().view(r, n // 32, 32) * _scales(s)[..., None]).view(r, n)


def _act(z, name):
    if name == "relu":
        return torch.where(z > 0, z, 0.0)
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        u = math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)
        return 0.5 * z * (1 + torch.tanh(u))
    return z


def _act_slope(z, name):
    if name == "relu":
        return (z > 0).float()
    if name == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    if name == "gelu":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def _linear_plain(s):
    c, ends = s["case"], s["ends"]
    kind, rows, k, n = TYPES[c["type"]], _rows_padded(c), c["inner"], c["outer"]
    groups = [(e, lo, hi) for e, (lo, hi) in enumerate(zip([0] + ends[:-1], ends)) if hi > lo]
    if c["way"] == "epilogue":
        dz = s["dy"].float()
        if c["activation"] != "none":
            dz = dz * _act_slope(s["z"].float(), c["activation"])
        dz[ends[-1]:] = 0
        dbias = torch.zeros(c["experts"] or 1, n, device="cuda")
        for e, lo, hi in groups:
            dbias[e] = dz[lo:hi].sum(0)
        return {"dz": dz.to(kind), "dbias": dbias}
    if c["way"] == "weights":
        dw = torch.zeros(c["experts"] or 1, n, k, device="cuda")
        for e, lo, hi in groups:
            parts = []
            for name, m in (("dz", n), ("x", k)):
                slab = s[name + "_s"][m * lo // 32:m * hi // 32]
                parts.append(_decode(s[name + "_q"][:, lo:hi], _unblocked(slab, m, (hi - lo) // 32)))
            dw[e] = parts[0] @ parts[1].t()
        if s["sum"] is None:
            return {"dw": dw.to(kind)}
        s["sum"].copy_(dw + s["sum"].float())
        return {"dw": s["sum"]}
    x = _decode(s["x_q"], _unblocked(s["x_s"], rows, k // 32))
    z = torch.zeros(rows, n, device="cuda")
    for e, lo, hi in groups:
        w = _decode(s["w_q"][e], _unblocked(s["w_s"][e * n * k // 32:(e + 1) * n * k // 32], n, k // 32))
        z[lo:hi] = x[lo:hi] @ w.t()
        if c["bias"]:
            z[lo:hi] += s["bias"][e]
    y = _act(z, c["activation"])
    if c["residual"]:
        y = y + s["residual"].float()
    y[ends[-1]:] = 0
    out = {"y": y.to(kind)}
    if c["keep"]:
        out["z"] = z.to(kind)
    return out


def _best_first(x, count):
    """The places of the `count` largest in each row, largest first, ties to the lowest place."""
    return torch.sort(x, dim=1, descending=True, stable=True).indices[:, :count]


def _route_plain(s):
    """The choice is made on scores in 64 bits: it hangs on their order alone."""
    c, x = s["case"], s["logits"].float()
    (t, e), k = x.shape, c["k"]
    routed = (x > -math.inf).any(1)
    if s["mask"] is not None:
        routed = routed & s["mask"]
    wide = x.double()
    if c["scores"] == "sigmoid":
        exact = 1 / (1 + torch.exp(-wide))
    else:
        z = torch.exp(wide - wide.amax(1, keepdim=True))
        exact = z / z.sum(1, keepdim=True)
    biased = torch.where((x > -math.inf) & routed[:, None], exact + s["bias"].double(), -math.inf)
    in_groups = torch.sort(biased.view(t, c["groups"], e // c["groups"]), dim=2, descending=True).values
    first, second = in_groups[..., 0], in_groups[..., min(1, e // c["groups"] - 1)]
    value = torch.where((second > -math.inf) & (e > c["groups"]), first + second, first)
    chosen = torch.zeros(t, c["groups"], dtype=torch.bool, device="cuda")
    chosen.scatter_(1, _best_first(value, c["best"]), True)
    allowed = chosen.repeat_interleave(e // c["groups"], 1)
    biased = torch.where(allowed, biased, -math.inf)
    ids = _best_first(biased, k)
    taken = biased.gather(1, ids) > -math.inf
    score = torch.where(routed[:, None], exact.float(), 0.0)
    picked = torch.where(taken, score.gather(1, ids), 0.0)
    total = picked.sum(1, keepdim=True) if c["renorm"] else torch.ones_like(picked[:, :1])
    w = torch.where(taken & (total > 0), picked / total, 0.0)
    counts = torch.bincount(ids[taken], minlength=e)
    n = routed.sum()
    share = e * counts.float() / (k * n.float() * n.float())
    every = score.sum(1, keepdim=True) if c["scores"] == "sigmoid" else torch.ones_like(score[:, :1])
    p = torch.where(every > 0, score / every, 0.0)
    loss = (share * p.sum(0)).sum()
    # gradients: of the scores first, then of the logits
    dw = torch.where(taken, s["dweights"], 0.0) * s["scale"]
    dpicked = dw
    if c["renorm"]:
        dpicked = torch.where(total > 0, (dw - (w * dw).sum(1, keepdim=True)) / total, 0.0)
    dscore = torch.zeros_like(score).scatter_add(1, ids, torch.where(taken, dpicked, 0.0))
    dp = (s["dloss"] * share)[None, :].expand(t, e)
    if c["scores"] == "sigmoid":
        dscore = dscore + torch.where(every > 0, (dp - (p * dp).sum(1, keepdim=True)) / every, 0.0)
        dx = dscore * score * (1 - score)
    else:
        dscore = dscore + dp
        dx = score * (dscore - (score * dscore).sum(1, keepdim=True))
    dx = torch.where(routed[:, None], dx, 0.0)
    return {"weights": w * s["scale"], "ids": torch.where(taken, ids, -1).int(), "counts": counts.int(), "loss": loss,
            "dlogits": dx.to(s["logits"].dtype)}


def _mixed(x):
    """A 32-bit mixing of numbers below 2^32, held in 64 bits: two rounds of shift,
    exclusive or and product with the fractional digits of the roots of 2 and 3."""
    x = x ^ (x >> 16)
    x = (x * 0x6A09E667) & 0xFFFFFFFF
    x = x ^ (x >> 15)
    x = (x * 0xBB67AE85) & 0xFFFFFFFF
    return x ^ (x >> 16)


def _random_bits(seed, step, at):
    """32 random bits of each place `at` in the moments, from the seed and the step."""
    one = torch.tensor([seed & 0xFFFFFFFF, seed >> 32, step & 0xFFFFFFFF], dtype=torch.int64, device="cuda")
    key = _mixed(_mixed(_mixed(one[0]) ^ one[1]) ^ one[2])
    return _mixed((at & 0xFFFFFFFF) ^ key ^ _mixed(at >> 32))


def _encode(x, u, keep):
    """E4M3 values and scale bytes of x [blocks, 32], rounded up with the probability of
    what lies above the value below (u uniform in [0, 1)).  keep: no other value becomes 0."""
    size = x.abs()
    bits = size.amax(1).view(torch.int32)
    scale = ((bits >> 23) - 8 + ((bits & 0x7FFFFF) > 0x600000).int()).clamp(min=0)
    size = size * ((254 - scale) << 23).view(torch.float32)[:, None]
    step = ((size.view(torch.int32) >> 23) - 127).clamp(min=-6) - 3  # the power of two of a last place
    q = torch.floor(size * ((127 - step) << 23).view(torch.float32) + u)
    if keep:
        q = torch.where((size > 0) & (q < 1), 1.0, q)
    q = q * ((127 + step) << 23).view(torch.float32)
    return torch.where(x < 0, -q, q).to(torch.float8_e4m3fn), scale.to(torch.uint8)


def _bytes(t):
    return t.view(torch.uint8)


def _adamw_plain(s):
    c = s["case"]
    (b1, b2), t = BETAS, s["step"]
    m_all, v_all, ms, vs = s["moments"]
    c1, c2 = 1 - b1**t, math.sqrt(1 - b2**t)
    for i, (p, g, at) in enumerate(zip(s["params"], s["grads"], s["starts"])):
        n = p.numel()
        blocks = (n + 31) // 32
        to, sc = slice(at, at + n), slice(at // 32, at // 32 + blocks)
        g = g.float() * s["grad_scale"]
        if c["bits"] == 32:
            m, v = m_all[to], v_all[to]
        else:
            whole = slice(at, at + 32 * blocks)
            m = _decode(m_all[whole].view(1, -1), ms[sc].view(1, -1)).view(-1)[:n]
            r = _decode(v_all[whole].view(1, -1), vs[sc].view(1, -1)).view(-1)[:n]
            v = r * r
        m = b1 * m + (1 - b1) * g
        v = b2 * v + (1 - b2) * (g * g)
        root = torch.sqrt(v)
        if c["bits"] == 32:
            m_all[to], v_all[to] = m, v
        else:
            place = torch.arange(at, at + 32 * blocks, device="cuda")
            bits = _random_bits(s["seed"], t, place).view(-1, 32)
            for x, low, q_all, s_all, keep in ((m, bits & 0xFFFF, m_all, ms, False), (root, bits >> 16, v_all, vs, True)):
                x = torch.nn.functional.pad(x, (0, 32 * blocks - n)).view(-1, 32)
                q, scale = _encode(x, low.float() / 65536, keep)
                q_all[whole], s_all[sc] = _bytes(q).view(-1), scale
        new = p.float() * (1 - LR * DECAY) - (LR / c1) * (m / (root / c2 + EPS))
        p.copy_(new)
        if c["copies"]:
            s["copies"][i].copy_(new)
    return _adamw_outputs(s)


def _adamw_outputs(s):
    m, v, ms, vs = s["moments"]
    out = {"params": s["all_params"], "m": m, "v": v}
    if ms is not None:  # the bytes as the values that they stand for: elements, and powers of two
        out = {"params": s["all_params"], "m": m.view(torch.float8_e4m3fn), "v": v.view(torch.float8_e4m3fn),
               "m_scale": ms, "v_scale": vs}
    if s["copies"] is not None:
        out["copies"] = s["all_copies"]
    return out


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    s, c = state, state["case"]
    if not own:
        return {"linear": _linear_plain, "route": _route_plain, "adamw": _adamw_plain}[c["op"]](s)
    import mx_block_quantization_gb300 as mxq
    if c["op"] == "linear":
        activation = None if c["activation"] == "none" else c["activation"]
        if c["way"] == "epilogue":
            dz, dbias = mxq.moe_linear_backward(s["dy"], s["z"], s["offs"], activation=activation)
            return {"dz": dz, "dbias": dbias.view(-1, c["outer"])}
        if c["way"] == "weights":
            dw = mxq.moe_weight_gradient(s["dz_q"], s["dz_s"], s["x_q"], s["x_s"], s["offs"], dtype=TYPES[c["type"]],
                                         out=None if s["sum"] is None else s["sum"] if c["experts"] else s["sum"][0],
                                         accumulate=s["sum"] is not None)
            return {"dw": dw.view(-1, c["outer"], c["inner"])}
        w, bias = s["w_q"], s["bias"]
        if not c["experts"]:
            w, bias = w[0], None if bias is None else bias[0]
        out = mxq.moe_linear(s["x_q"], s["x_s"], w, s["w_s"], s["offs"], bias=bias, activation=activation,
                             residual=s["residual"], preactivation=c["keep"], dtype=TYPES[c["type"]])
        return {"y": out[0], "z": out[1]} if c["keep"] else {"y": out}
    if c["op"] == "route":
        how = dict(bias=s["bias"], scores=c["scores"], groups=c["groups"], best_groups=c["best"], mask=s["mask"],
                   renorm=c["renorm"], scale=s["scale"])
        r = mxq.moe_route_groups(s["logits"], c["k"], **how)
        dlogits = mxq.moe_route_groups_backward(s["logits"], r, s["dweights"], s["dloss"], mask=s["mask"],
                                                scores=c["scores"], renorm=c["renorm"], scale=s["scale"])
        return {"weights": r.weights, "ids": r.ids, "counts": r.counts, "loss": r.loss, "dlogits": dlogits}
    mxq.adamw_step(s["params"], s["grads"], mxq.Moments(*s["moments"]), s["step"], lr=LR, betas=BETAS, eps=EPS,
                   weight_decay=DECAY, grad_scale=s["grad_scale"], copies=s["copies"], seed=s["seed"])
    return _adamw_outputs(s)


# ---------------------------------------------------------------------------
# from the definitions, in 64 bits
# ---------------------------------------------------------------------------

def _e4m3_table():
    """The value of each E4M3 byte: sign, 4 bits of exponent (bias 7), 3 of mantissa."""
    values = []
    for b in range(256):
        e, f = b >> 3 & 15, b & 7
        v = f * 2.0**-9 if e == 0 else (8 + f) * 2.0**(e - 10)
        values.append(math.nan if b & 127 == 127 else -v if b & 128 else v)
    return torch.tensor(values, dtype=torch.float64, device="cuda")


def _values64(q, s, first=0):
    """Values of E4M3 bytes [R, C]; the scale of (r, c) is looked up in the blocked layout."""
    r, n = q.shape
    i, j = torch.arange(r, device="cuda")[:, None], torch.arange(n // 32, device="cuda")[None, :]
    at = first + ((i // 128) * (n // 128) + j // 4) * 512 + (i % 32) * 16 + (i % 128) // 32 * 4 + j % 4
    scale = torch.pow(2.0, s[at].double() - 127)
    return _e4m3_table()[q.long()] * scale.repeat_interleave(32, 1)


def _act64(z, name):
    if name == "relu":
        return torch.relu(z)
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        # 0.5 (1 + tanh u) is the logistic function of 2u
        return z * torch.sigmoid(math.sqrt(8 / math.pi) * z * (1 + 0.044715 * z**2))
    return z


def _linear_exact(s):
    c, ends = s["case"], s["ends"]
    rows, k, n = _rows_padded(c), c["inner"], c["outer"]
    if c["way"] != "epilogue" and 2 * ends[-1] * k * n > 1.6e13:
        return None
    begins = [0] + ends[:-1]
    if c["way"] == "epilogue":
        z = s["z"].double().requires_grad_()
        y = _act64(z, c["activation"])
        y.backward(s["dy"].double())
        dz = z.grad
        dz[ends[-1]:] = 0
        group = torch.repeat_interleave(torch.arange(len(ends), device="cuda"),
                                        torch.tensor([hi - lo for lo, hi in zip(begins, ends)], device="cuda"))
        dbias = torch.zeros(len(ends), n, dtype=torch.float64, device="cuda")
        dbias.index_add_(0, group, dz[:ends[-1]])
        return {"dz": dz, "dbias": dbias}
    if c["way"] == "weights":
        dw = torch.zeros(len(ends), n, k, dtype=torch.float64, device="cuda")
        for e, (lo, hi) in enumerate(zip(begins, ends)):
            if hi > lo:
                dw[e] = torch.einsum("nm,km->nk", _values64(s["dz_q"][:, lo:hi], s["dz_s"], n * lo // 32),
                                     _values64(s["x_q"][:, lo:hi], s["x_s"], k * lo // 32))
        return {"dw": dw if s["sum"] is None else dw + s["sum"].double()}
    x = _values64(s["x_q"], s["x_s"])
    z = torch.zeros(rows, n, dtype=torch.float64, device="cuda")
    for e, (lo, hi) in enumerate(zip(begins, ends)):
        if hi > lo:
            z[lo:hi] = torch.einsum("mk,nk->mn", x[lo:hi], _values64(s["w_q"][e], s["w_s"], e * n * k // 32))
            if c["bias"]:
                z[lo:hi] += s["bias"][e].double()
    y = _act64(z, c["activation"])
    if c["residual"]:
        y = y + s["residual"].double()
    y[ends[-1]:] = 0
    return {"y": y, "z": z} if c["keep"] else {"y": y}


def _route_exact(s):
    """Balance loss and weights as a function of the logits, differentiated by autograd;
    the choice by a search for the largest that is left."""
    c, k, e = s["case"], s["case"]["k"], s["case"]["experts"]
    keep = torch.isfinite(s["logits"].double()).any(1)
    if s["mask"] is not None:
        keep &= s["mask"]
    at = keep.nonzero()[:, 0]
    x = s["logits"].double()[at].requires_grad_()
    score = torch.sigmoid(x) if c["scores"] == "sigmoid" else torch.softmax(x, 1)
    left = score.detach() + s["bias"].double()
    groups = left.view(at.numel(), c["groups"], -1)
    value = torch.topk(groups, min(2, groups.shape[2]), dim=2).values.sum(2)
    allowed = torch.zeros_like(value, dtype=torch.bool)
    for _ in range(c["best"]):
        g = value.argmax(1, keepdim=True)
        allowed.scatter_(1, g, True)
        value.scatter_(1, g, -math.inf)
    left = torch.where(allowed[..., None], groups, -math.inf).view(at.numel(), e)
    ids = []
    for _ in range(k):
        best = left.max(1, keepdim=True).values
        i = torch.where(left == best, torch.arange(e, device="cuda"), e).amin(1, keepdim=True)
        ids.append(i)
        left.scatter_(1, i, -math.inf)
    ids = torch.cat(ids, 1)
    w = score.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    w = w * s["scale"]
    p = score / score.sum(1, keepdim=True)
    counts = torch.zeros(e, dtype=torch.float64, device="cuda")
    counts.index_add_(0, ids.reshape(-1), torch.ones(ids.numel(), dtype=torch.float64, device="cuda"))
    loss = e * ((counts / (k * at.numel())) * p.mean(0)).sum()
    ((w * s["dweights"].double()[at]).sum() + s["dloss"].double() * loss).backward()
    weights = torch.zeros(c["tokens"], k, dtype=torch.float64, device="cuda")
    all_ids = torch.full((c["tokens"], k), -1, dtype=torch.int32, device="cuda")
    dlogits = torch.zeros(c["tokens"], e, dtype=torch.float64, device="cuda")
    weights[at], all_ids[at], dlogits[at] = w.detach(), ids.int(), x.grad
    return {"weights": weights, "ids": all_ids, "counts": counts.int(), "loss": loss.detach(), "dlogits": dlogits}


def _adamw_exact(s):
    """The step on all tensors at once; moments in MXFP8 are rounded at random, so that
    their bytes have no value of their own here."""
    c = s["case"]
    m, v, ms, vs = s["moments"]
    if ms is None:
        m, v = m.double(), v.double()
    else:
        table = _e4m3_table()
        m = table[m.long()] * torch.pow(2.0, ms.double() - 127).repeat_interleave(32)
        v = (table[v.long()] * torch.pow(2.0, vs.double() - 127).repeat_interleave(32)) ** 2
    total = m.numel()
    inside = torch.zeros(total, dtype=torch.bool, device="cuda")
    g = torch.zeros(total, dtype=torch.float64, device="cuda")
    for t, at in zip(s["grads"], s["starts"]):
        inside[at:at + t.numel()] = True
        g[at:at + t.numel()] = t.double()
    g *= s["grad_scale"].double()
    (b1, b2), t = BETAS, s["step"]
    m, v = torch.lerp(g, m, b1), torch.lerp(g**2, v, b2)
    p = s["all_params"].double()
    new = p - LR * (DECAY * p + m / (1 - b1**t) / ((v / (1 - b2**t)).sqrt() + EPS))
    new = torch.where(inside, new, p)
    out = {"params": new, "m": m, "v": v} if ms is None else {"params": new, "m": None, "v": None, "m_scale": None, "v_scale": None}
    if c["copies"]:
        out["copies"] = torch.where(inside, new, s["all_copies"].double())
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"linear": _linear_exact, "route": _route_exact, "adamw": _adamw_exact}[case["op"]](s)
