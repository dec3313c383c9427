"""The training operators around the MXFP8 cast, as cases to measure and compare.

Four operators of a mixture-of-experts training step, each in its plain form
(elementary torch operations in 32 bits, rounded once at the end) and through
the package's own calls:

* route          router logits -> the k experts of each token, their weights, the
                 count of each expert and the balance loss; then the gradient of the
                 logits from those of the weights and of the loss.
* exchange       tokens to the 128-row aligned expert groups that the grouped cast
                 takes (offs, slots, source, rows) and the experts' outputs back to
                 the tokens; or the gradients of both.
* embedding      scaled lookup, or the gradient of the table.
* orthogonalize  Newton-Schulz products of a momentum (or of a stack of them).
"""
import math

import torch

own = False

COEFFICIENTS = (3.4445, -4.775, 2.0315)
STEPS = 5
EPS = 1e-7
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # a micro-batch of a few tokens: latency of the calls counts
        {"name": "route small", "op": "route", "tokens": 32, "experts": 64, "k": 8, "type": "f32",
         "renorm": True, "masked": 0.0, "pad": 0},
        # the routing that gives the grouped cast its 57344 routed rows in 64 groups
        {"name": "route step", "op": "route", "tokens": 7168, "experts": 64, "k": 8, "type": "bf16",
         "renorm": True, "masked": 0.0, "pad": 0},
        # a long packed batch with padding tokens, an odd number of experts, strided logits
        {"name": "route long", "op": "route", "tokens": 131071, "experts": 250, "k": 6, "type": "f32",
         "renorm": False, "masked": 0.1, "pad": 6},
        # few tokens, most groups with one to four rows: nearly all of the rows are padding
        {"name": "exchange small", "op": "exchange", "way": "forward", "tokens": 32, "width": 1024,
         "experts": 64, "k": 8, "type": "bf16", "dropped": 0.0},
        # the grouped cast's workload: 57344 routed rows of width 7168 in 64 groups
        {"name": "exchange step", "op": "exchange", "way": "forward", "tokens": 7168, "width": 7168,
         "experts": 64, "k": 8, "type": "bf16", "dropped": 0.0},
        # gradients in fp32 at sizes that are no powers of two, with tokens that no expert takes
        {"name": "exchange gradient", "op": "exchange", "way": "gradient", "tokens": 10007, "width": 2050,
         "experts": 96, "k": 3, "type": "f32", "dropped": 0.05},
        # the tokens of one decoding step: latency
        {"name": "lookup small", "op": "embedding", "way": "lookup", "tokens": 8, "vocabulary": 32768,
         "width": 4096, "type": "bf16", "ids": "i64", "padding": False, "pad": 0},
        # the table's gradient of a training step: most of the time is writing the table
        {"name": "table gradient", "op": "embedding", "way": "gradient", "tokens": 16384,
         "vocabulary": 131072, "width": 4096, "type": "bf16", "ids": "i64", "padding": False, "pad": 0},
        # odd width, odd vocabulary, padding tokens left out, strided gradient rows
        {"name": "table gradient odd", "op": "embedding", "way": "gradient", "tokens": 40009,
         "vocabulary": 50021, "width": 1001, "type": "f32", "ids": "i32", "padding": True, "pad": 3},
        # one small matrix of odd sizes: a chain of small dependent products
        {"name": "orthogonalize small", "op": "orthogonalize", "batch": 1, "rows": 200, "columns": 333,
         "type": "f32", "pad": 0},
        # one projection of 64 experts, taller than wide
        {"name": "orthogonalize experts", "op": "orthogonalize", "batch": 64, "rows": 1024,
         "columns": 512, "type": "bf16", "pad": 0},
        # one large projection
        {"name": "orthogonalize large", "op": "orthogonalize", "batch": 1, "rows": 4096,
         "columns": 8192, "type": "f32", "pad": 0},
    ]


def draw(rng):
    def log(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["route", "exchange", "embedding", "orthogonalize"])
    kind = rng.choice(["f32", "bf16"])
    if op == "route":
        experts = log(2, 384)
        return {"op": op, "tokens": min(log(1, 131071), 131071 * 250 // experts), "experts": experts,
                "k": rng.randint(1, min(8, experts)), "type": kind, "renorm": rng.random() < 0.5,
                "masked": rng.choice([0.0, 0.1, 0.5]), "pad": rng.choice([0, 0, 1, 8])}
    if op == "exchange":
        experts, width = log(2, 256), log(64, 7168)
        k = rng.randint(1, min(8, experts))
        if rng.random() < 0.7:
            width = max(64, width // 8 * 8)
        most = 4300 * 7168 * 8 // (2 if kind == "f32" else 1) // (k * width)
        return {"op": op, "way": rng.choice(["forward", "gradient"]), "tokens": min(log(1, 16384), most),
                "width": width, "experts": experts, "k": k, "type": kind,
                "dropped": rng.choice([0.0, 0.05])}
    if op == "embedding":
        vocabulary, width = log(128, 131072), log(16, 4096)
        if rng.random() < 0.7:
            width = max(16, width // 8 * 8)
        if kind == "f32":
            vocabulary = max(128, vocabulary // 2)
        return {"op": op, "way": rng.choice(["lookup", "gradient"]), "tokens": log(1, 65536 if width <= 2048 else 16384),
                "vocabulary": vocabulary, "width": width, "type": kind, "ids": rng.choice(["i32", "i64"]),
                "padding": rng.random() < 0.3, "pad": rng.choice([0, 0, 0, 8, 3])}
    rows, columns = log(16, 4096), log(16, 8192)
    if rng.random() < 0.5:
        rows, columns = columns, rows
    if rng.random() < 0.5:
        rows, columns = max(16, rows // 64 * 64), max(16, columns // 64 * 64)
    most = 0.5 * _orthogonal_flops(4096, 8192) / _orthogonal_flops(rows, columns)
    batch = 1 if rng.random() < 0.5 else max(1, min(log(1, 64), int(most), (1 << 26) // (rows * columns)))
    return {"op": op, "batch": batch, "rows": rows, "columns": columns, "type": kind,
            "pad": rng.choice([0, 0, 0, 8, 5])}


def _groups_rows(tokens, k, experts):
    """Rows that hold any routing of tokens*k rows in groups of whole 128 rows."""
    routed = tokens * k
    return (routed + 127 * min(experts, routed)) // 128 * 128


def _orthogonal_flops(rows, columns):
    """A product with its own transpose and the square of a symmetric matrix have
    one triangle to compute; the third product has every element."""
    r, c = min(rows, columns), max(rows, columns)
    return STEPS * (r * r * c + r * r * r + 2 * r * r * c)


def work(case):
    c = case
    if c["op"] == "orthogonalize":
        n = c["batch"] * c["rows"] * c["columns"]
        return {"bytes": n * (4 if c["type"] == "f32" else 2) + 2 * n,
                "flops": c["batch"] * _orthogonal_flops(c["rows"], c["columns"])}
    e, t = (4 if c["type"] == "f32" else 2), c["tokens"]
    if c["op"] == "route":
        n, s = t * c["experts"], t * c["k"]
        # logits in, their gradient out; weights and ids out, the weights' gradient in
        return {"bytes": 2 * n * e + s * 12 + c["experts"] * 4, "flops": 20 * n}
    d = c["width"]
    if c["op"] == "exchange":
        m, s = _groups_rows(t, c["k"], c["experts"]), t * c["k"]
        live = s * (1 - c["dropped"])
        if c["way"] == "forward":  # x in, rows out; the experts' rows in, y out
            return {"bytes": e * d * (t + m + live + t) + s * 12 + m * 4 + c["experts"] * 4, "flops": 2 * s * d}
        # dy and the experts' rows in, their gradient out; the gradient of the dispatched rows in, dx out
        return {"bytes": e * d * (t + live + m + live + t) + s * 16 + m * 4, "flops": 4 * s * d}
    i = 4 if c["ids"] == "i32" else 8
    if c["way"] == "lookup":
        return {"bytes": 2 * t * d * e + t * i, "flops": t * d}
    return {"bytes": t * d * e + c["vocabulary"] * d * e + t * i, "flops": t * d}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _normal(shape, g, kind="f32", scale=1.0, pad=0):
    """Normal values; with `pad`, rows that lie further apart than they are long."""
    *lead, n = shape
    x = torch.randn(*lead, n + pad, generator=g, device="cuda") * scale
    return x.to(TYPES[kind])[..., :n]


def _routing(tokens, experts, k, g):
    """k different experts for each token, some experts taken far more often than others."""
    liked = torch.randn(experts, generator=g, device="cuda")
    return torch.topk(torch.randn(tokens, experts, generator=g, device="cuda") + liked, k, dim=1)


def _plan_of(ids, experts):
    """offs, slots and source of a routing, from their definition."""
    tokens, k = ids.shape
    flat = ids.reshape(-1).long()
    live = flat >= 0
    counts = torch.bincount(flat[live], minlength=experts)
    ends = torch.cumsum((counts + 127) // 128 * 128, 0)
    begins = ends - (counts + 127) // 128 * 128
    order = torch.argsort(torch.where(live, flat, experts), stable=True)
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=ids.device)
    before = torch.cumsum(counts, 0) - counts
    at = flat.clamp(min=0)
    slots = torch.where(live, begins[at] + place - before[at], -1)
    rows = _groups_rows(tokens, k, experts)
    source = torch.full((rows + 1,), -1, dtype=torch.int32, device=ids.device)
    source[torch.where(live, slots, rows)] = torch.arange(flat.numel(), device=ids.device, dtype=torch.int32)
    return ends.int(), slots.reshape(tokens, k).int(), source[:rows].contiguous()


def prepare(case, seed):
    c, g = case, torch.Generator(device="cuda").manual_seed(seed)
    if c["op"] == "route":
        t, e = c["tokens"], c["experts"]
        liked = torch.randn(e, generator=g, device="cuda")
        logits = torch.randn(t, e + c["pad"], generator=g, device="cuda") * 1.5
        logits[:, :e] += liked
        mask = None
        if c["masked"]:
            mask = torch.rand(t, generator=g, device="cuda") >= c["masked"]
            mask[0] = True
        return {"case": c, "logits": logits.to(TYPES[c["type"]])[:, :e], "mask": mask,
                "dweights": torch.randn(t, c["k"], generator=g, device="cuda") * 0.1,
                "dloss": torch.rand((), generator=g, device="cuda") * 0.01 + 0.005}
    if c["op"] == "exchange":
        t, d, e, k = c["tokens"], c["width"], c["experts"], c["k"]
        best, ids = _routing(t, e, k, g)
        ids = ids.int()
        if c["dropped"]:
            gone = torch.rand(t, generator=g, device="cuda") < c["dropped"]
            ids = torch.where(gone[:, None], -1, ids)
        m = _groups_rows(t, k, e)
        s = {"case": c, "ids": ids.contiguous(), "weights": torch.softmax(best, 1)}
        s["experts_rows"] = _normal((m, d), g, c["type"], 0.5)
        if c["way"] == "forward":
            s["x"] = _normal((t, d), g, c["type"])
        else:
            s["plan"] = _plan_of(ids, e)
            s["dy"] = _normal((t, d), g, c["type"], 0.1)
            s["dispatched"] = _normal((m, d), g, c["type"], 0.1)
        return s
    if c["op"] == "embedding":
        t, v, d = c["tokens"], c["vocabulary"], c["width"]
        # word frequencies fall off as one over the rank; ranks are spread over the table
        rank = torch.exp(torch.rand(t, generator=g, device="cuda", dtype=torch.float64) * math.log(v)).long() - 1
        ids = (rank.clamp(0, v - 1) * 7919 + 13) % v
        ids = ids.to(torch.int32 if c["ids"] == "i32" else torch.int64)
        s = {"case": c, "ids": ids, "scale": math.sqrt(d), "padding": 13 % v if c["padding"] else None}
        if c["way"] == "lookup":
            s["table"] = _normal((v, d), g, c["type"], 0.02, c["pad"])
        else:
            s["dy"] = _normal((t, d), g, c["type"], 0.01, c["pad"])
        return s
    b, r, n = c["batch"], c["rows"], c["columns"]
    few = max(1, min(r, n) // 16)
    # a momentum: a few strong directions over a floor of noise
    x = torch.randn(b, r, few, generator=g, device="cuda") @ torch.randn(b, few, n, generator=g, device="cuda")
    x = x * (1e-3 / math.sqrt(few))
    x = torch.nn.functional.pad(x, (0, c["pad"])) + 1e-3 * torch.randn(b, r, n + c["pad"], generator=g, device="cuda")
    x = x.to(TYPES[c["type"]])[..., :n]
    return {"case": c, "momentum": x if b > 1 else x[0]}


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _route_plain(s):
    c, x = s["case"], s["logits"].float()
    (t, e), k = x.shape, c["k"]
    routed = (x > -math.inf).any(1)
    if s["mask"] is not None:
        routed = routed & s["mask"]
    top = torch.where(routed, x.max(1).values, 0.0)
    z = torch.exp(x - top[:, None])
    p = torch.where(routed[:, None], z / z.sum(1, keepdim=True), 0.0)
    best, ids = torch.sort(x, dim=1, descending=True, stable=True)
    taken = routed[:, None] & (best[:, :k] > -math.inf)
    ids = ids[:, :k]
    w = torch.where(taken, p.gather(1, ids), 0.0)
    if c["renorm"]:
        w = torch.where(taken, w / w.sum(1, keepdim=True), 0.0)
    counts = torch.bincount(ids[taken], minlength=e)
    n = routed.sum()
    share = e * counts.float() / (k * n.float() * n.float())
    loss = (share * p.sum(0)).sum()
    # gradients
    dw = torch.where(taken, s["dweights"], 0.0)
    dp = (s["dloss"] * share)[None, :].expand(t, e)
    dx = p * (dp - (p * dp).sum(1, keepdim=True))
    if c["renorm"]:
        dx = dx.scatter_add(1, ids, w * (dw - (w * dw).sum(1, keepdim=True)))
    else:
        chosen = torch.zeros_like(p).scatter_add(1, ids, dw)
        dx = dx + p * (chosen - (p * chosen).sum(1, keepdim=True))
    return {"weights": w, "ids": torch.where(taken, ids, -1).int(), "counts": counts.int(),
            "loss": loss, "dlogits": dx.to(s["logits"].dtype)}


def _gather_rows(rows, index):
    """rows[index] in 32 bits, zero where the index is negative."""
    return torch.where((index >= 0)[..., None], rows[index.clamp(min=0).long()].float(), 0.0)


def _exchange_plain(s):
    c, kind = s["case"], s["experts_rows"].dtype
    k = c["k"]
    if c["way"] == "forward":
        offs, slots, source = _plan_of(s["ids"], c["experts"])
        token = torch.where(source >= 0, source // k, -1)
        rows = torch.where((token >= 0)[:, None], s["x"][token.clamp(min=0).long()], 0)
        y = torch.zeros(s["x"].shape, device="cuda")
        for j in range(k):
            y += s["weights"][:, j, None] * _gather_rows(s["experts_rows"], slots[:, j])
        return {"offs": offs, "slots": slots, "source": source, "rows": rows, "y": y.to(kind)}
    offs, slots, source = s["plan"]
    token = torch.where(source >= 0, source // k, -1)
    w = s["weights"].reshape(-1)[source.clamp(min=0).long()]
    drows = (w[:, None] * _gather_rows(s["dy"], token)).to(kind)
    dy, dx = s["dy"].float(), torch.zeros(s["dy"].shape, device="cuda")
    dweights = torch.empty_like(s["weights"])
    for j in range(k):
        dweights[:, j] = (dy * _gather_rows(s["experts_rows"], slots[:, j])).sum(1)
        dx += _gather_rows(s["dispatched"], slots[:, j])
    return {"drows": drows, "dweights": dweights, "dx": dx.to(kind)}


def _embedding_plain(s):
    c, ids = s["case"], s["ids"].long()
    if c["way"] == "lookup":
        return {"y": (s["table"][ids].float() * s["scale"]).to(s["table"].dtype)}
    dy = s["dy"].float() * s["scale"]
    if s["padding"] is not None:
        dy = torch.where((ids == s["padding"])[:, None], 0.0, dy)
    table = torch.zeros(c["vocabulary"], c["width"], device="cuda")
    table.index_add_(0, ids, dy)
    return {"dtable": table.to(s["dy"].dtype)}


def _orthogonalize_plain(s):
    a, b, c = COEFFICIENTS
    x = s["momentum"].float()
    tall = x.shape[-2] > x.shape[-1]
    if tall:
        x = x.mT
    x = x / (x.square().sum((-2, -1), keepdim=True).sqrt() + EPS)
    for _ in range(STEPS):
        square = x @ x.mT
        x = a * x + (b * square + c * (square @ square)) @ x
    return {"update": (x.mT if tall else x).to(torch.bfloat16)}


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    s, c = state, state["case"]
    if not own:
        plain = {"route": _route_plain, "exchange": _exchange_plain, "embedding": _embedding_plain,
                 "orthogonalize": _orthogonalize_plain}
        return plain[c["op"]](s)
    import mx_block_quantization_gb300 as mxq
    if c["op"] == "route":
        r = mxq.moe_route(s["logits"], c["k"], mask=s["mask"], renorm=c["renorm"])
        dlogits = mxq.moe_route_backward(s["logits"], r, s["dweights"], s["dloss"], mask=s["mask"],
                                         renorm=c["renorm"])
        return {"weights": r.weights, "ids": r.ids, "counts": r.counts, "loss": r.loss, "dlogits": dlogits}
    if c["op"] == "exchange":
        if c["way"] == "forward":
            plan = mxq.moe_plan(s["ids"], c["experts"])
            rows = mxq.moe_dispatch(s["x"], plan)
            y = mxq.moe_combine(s["experts_rows"], plan, s["weights"])
            return {"offs": plan.offs, "slots": plan.slots, "source": plan.source, "rows": rows, "y": y}
        plan = mxq.MoePlan(*s["plan"])
        drows, dweights = mxq.moe_combine_backward(s["dy"], s["experts_rows"], plan, s["weights"])
        return {"drows": drows, "dweights": dweights, "dx": mxq.moe_combine(s["dispatched"], plan)}
    if c["op"] == "embedding":
        if c["way"] == "lookup":
            return {"y": mxq.embedding(s["ids"], s["table"], scale=s["scale"])}
        return {"dtable": mxq.embedding_backward(s["ids"], s["dy"], c["vocabulary"], scale=s["scale"],
                                                 padding_idx=s["padding"])}
    return {"update": mxq.orthogonalize(s["momentum"], steps=STEPS, coefficients=COEFFICIENTS, eps=EPS)}


# ---------------------------------------------------------------------------
# from the definitions, in 64 bits
# ---------------------------------------------------------------------------

def _route_exact(s):
    """Balance loss and weights as a function of the logits, differentiated by autograd."""
    c, k = s["case"], s["case"]["k"]
    e = c["experts"]
    keep = torch.isfinite(s["logits"].double()).any(1)
    if s["mask"] is not None:
        keep &= s["mask"]
    at = keep.nonzero()[:, 0]
    x = s["logits"].double()[at].requires_grad_()
    ids = torch.argsort(-x.detach(), dim=1, stable=True)[:, :k]
    logp = torch.log_softmax(x, 1)
    chosen = logp.gather(1, ids)
    w = torch.softmax(chosen, 1) if c["renorm"] else chosen.exp()
    counts = torch.zeros(e, dtype=torch.float64, device="cuda")
    counts.index_add_(0, ids.reshape(-1), torch.ones(ids.numel(), dtype=torch.float64, device="cuda"))
    loss = e * ((counts / (k * at.numel())) * logp.exp().mean(0)).sum()
    ((w * s["dweights"].double()[at]).sum() + s["dloss"].double() * loss).backward()
    weights = torch.zeros(c["tokens"], k, dtype=torch.float64, device="cuda")
    all_ids = torch.full((c["tokens"], k), -1, dtype=torch.int32, device="cuda")
    dlogits = torch.zeros(c["tokens"], e, dtype=torch.float64, device="cuda")
    weights[at], all_ids[at], dlogits[at] = w.detach(), ids.int(), x.grad
    return {"weights": weights, "ids": all_ids, "counts": counts.int(), "loss": loss.detach(), "dlogits": dlogits}


def _exchange_exact(s):
    """The exchange as sums over the list of (token, choice, expert) in the order of the groups."""
    c, ids = s["case"], s["ids"].cpu()
    t, k, d = c["tokens"], c["k"], c["width"]
    groups = [[] for _ in range(c["experts"])]
    for i, expert in enumerate(ids.reshape(-1).tolist()):
        if expert >= 0:
            groups[expert].append(i)
    source, ends = [], []
    for group in groups:
        source += group + [-1] * (-len(group) % 128)
        ends.append(len(source))
    source += [-1] * (_groups_rows(t, k, c["experts"]) - len(source))
    slots = [-1] * (t * k)
    for slot, i in enumerate(source):
        if i >= 0:
            slots[i] = slot
    slots = torch.tensor(slots, dtype=torch.int32)
    source = torch.tensor(source, dtype=torch.int32)
    at = (slots >= 0).nonzero()[:, 0].cuda()
    token, slot = at // k, slots.cuda()[at].long()
    w = s["weights"].double().reshape(-1)[at]
    if c["way"] == "forward":
        rows = torch.zeros(source.numel(), d, dtype=s["x"].dtype, device="cuda")
        rows[slot] = s["x"][token]
        y = torch.zeros(t, d, dtype=torch.float64, device="cuda")
        for j in range(k):  # choice by choice: the rows of a token are added one at a time
            part = at % k == j
            y[token[part]] += w[part, None] * s["experts_rows"][slot[part]].double()
        return {"offs": torch.tensor(ends, dtype=torch.int32), "slots": slots.reshape(t, k), "source": source,
                "rows": rows, "y": y}
    drows = torch.zeros(source.numel(), d, dtype=torch.float64, device="cuda")
    drows[slot] = w[:, None] * s["dy"].double()[token]
    dweights = torch.zeros(t * k, dtype=torch.float64, device="cuda")
    dweights[at] = torch.einsum("nd,nd->n", s["dy"].double()[token], s["experts_rows"].double()[slot])
    dx = torch.zeros(t, d, dtype=torch.float64, device="cuda")
    for j in range(k):
        part = at % k == j
        dx[token[part]] += s["dispatched"][slot[part]].double()
    return {"drows": drows, "dweights": dweights.reshape(t, k), "dx": dx}


def _embedding_exact(s):
    c, ids = s["case"], s["ids"].long()
    if c["way"] == "lookup":
        return {"y": s["scale"] * s["table"].double().index_select(0, ids)}
    # rows in the order of their ids, summed by differences of the places where an id ends
    order = torch.argsort(ids, stable=True)
    if s["padding"] is not None:
        order = order[ids[order] != s["padding"]]
    out = torch.zeros(c["vocabulary"], c["width"], dtype=torch.float64, device="cuda")
    if order.numel():
        which, lengths = torch.unique_consecutive(ids[order], return_counts=True)
        out[which] = torch.segment_reduce(s["scale"] * s["dy"][order].double(), "sum", lengths=lengths)
    return {"dtable": out}


def _orthogonalize_exact(s):
    a, b, c = COEFFICIENTS
    x = s["momentum"].double()
    x = x / (torch.linalg.norm(x.flatten(-2), dim=-1)[..., None, None] + EPS)
    wide = x.shape[-2] <= x.shape[-1]
    for _ in range(STEPS):
        gram = x @ x.mT if wide else x.mT @ x
        one = torch.eye(gram.shape[-1], dtype=torch.float64, device="cuda")
        poly = a * one + gram @ (b * one + c * gram)
        x = poly @ x if wide else x @ poly
    return {"update": x}


def exact(case, seed):
    s = prepare(case, seed)
    how = {"route": _route_exact, "exchange": _exchange_exact, "embedding": _embedding_exact,
           "orthogonalize": _orthogonalize_exact}
    return how[case["op"]](s)
