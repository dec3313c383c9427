"""Operators of a mixture-of-experts training step around the MXFP8 cast.

Routing with its balance loss (:func:`moe_route`, :func:`moe_route_groups`), the
exchange of rows with the 128-row expert groups that :func:`quantize_2d_dual` takes
(:func:`moe_plan`, :func:`moe_dispatch`, :func:`moe_combine`), the experts' products on
what it gives (:func:`moe_linear`, :func:`moe_weight_gradient`,
:func:`moe_linear_backward`), the embedding table (:func:`embedding`) and their
gradients, each a call of its own, and what moves the parameters
(:func:`orthogonalize`, :func:`adamw_step`).  The functions
marshal torch CUDA tensors into the C ABI of ``include/mxq.h``, which states
each operation; there is no CPU path.

Matrices may have strided rows (unit column stride).  With ``stream`` a call runs
on that stream, and the outputs and workspaces that it allocates belong to it;
it has to be a stream of the tensors' device.  Otherwise the call runs on the current
stream of that device.
"""
from __future__ import annotations

import ctypes
from contextlib import nullcontext
from operator import index
from typing import NamedTuple, Optional

import torch

from . import BF16, EBADSHAPE, F32, OK, MxqError, lib

_CODES = {torch.float32: F32, torch.bfloat16: BF16}


class Routing(NamedTuple):
    weights: torch.Tensor  # float32 [T, k]
    ids: torch.Tensor      # int32 [T, k], -1 where there is no expert
    counts: torch.Tensor   # int32 [E]
    loss: torch.Tensor     # float32 []
    routed: torch.Tensor   # int32 []: tokens that take part


class MoePlan(NamedTuple):
    offs: torch.Tensor    # int32 [E]: cumulative group ends, multiples of 128
    slots: torch.Tensor   # int32 [T, k]: row of each assignment, -1 for none
    source: torch.Tensor  # int32 [M]: assignment of each row, -1 for none


class Moments(NamedTuple):
    m: torch.Tensor                   # float32, or uint8 E4M3 [total]
    v: torch.Tensor                   # float32; in 8 bits the bytes of its root
    m_scale: Optional[torch.Tensor]   # None, or uint8 E8M0 [total / 32]
    v_scale: Optional[torch.Tensor]


def _count(value, what):
    """A count as the C entries take it; ctypes would cut it to its lowest bits."""
    value = index(value)
    if -0x80000000 <= value <= 0x7FFFFFFF:
        return value
    raise MxqError(EBADSHAPE, what)


def _code(t, name):
    code = _CODES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be float32 or bfloat16")
    return code


def _matrix(t, name, rows=None, cols=None, device=None):
    """Row pitch of a 2-D CUDA tensor with unit column stride."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (no CPU path)")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    m, n = t.shape
    if (rows is not None and m != rows) or (cols is not None and n != cols):
        raise ValueError(f"{name} must be [{m if rows is None else rows}, {n if cols is None else cols}]")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}")
    if m <= 1 or n == 0:
        if n > 1 and t.stride(1) != 1:
            raise ValueError(f"{name} must have unit column stride")
        return max(n, 1)
    ld = t.stride(0)
    if (n > 1 and t.stride(1) != 1) or ld < n:
        raise ValueError(f"{name} must have unit column stride and rows that do not overlap")
    return ld


def _rows_of(t, name, T, D):
    """[..., D] as a matrix [T, D] of the same memory."""
    if t.dim() == 2:
        return t  # as it is: another view takes 2 us
    if T == 0 or D == 0:
        return t.reshape(T, D)
    try:
        return t.view(T, D)
    except RuntimeError:
        raise ValueError(f"{name} must have rows a fixed distance apart") from None


def _flat(t, name, dtype, shape, device):
    """A contiguous CUDA tensor of one type and shape."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (no CPU path)")
    if t.dtype != dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {list(shape)} on {device}")
    return t.data_ptr()


def _mask_pointer(mask, tokens, device):
    return _flat(mask, "mask", torch.uint8 if mask.dtype == torch.uint8 else torch.bool, (tokens,), device)


def _elsewhere(device, stream):
    """None when a call on `device` may run as things are, else the context in
    which its allocations and launches belong to its device and stream."""
    if stream is not None:
        if stream.device != device:
            raise ValueError(f"stream must be one of {device}, where the tensors are, not of {stream.device}")
        return torch.cuda.stream(stream)
    return None if torch.cuda.current_device() == device.index else torch.cuda.device(device)


# the handle of a device's current stream; the public call builds a Stream object
# around it, which takes as long as a launch
_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _workspace(size, what, device):
    """(tensor, pointer) of a call's workspace of the size the library asks for."""
    if size <= 0:
        if size < 0:
            raise MxqError(int(size), what)
        return None, None
    t = torch.empty(size, dtype=torch.uint8, device=device)
    return t, t.data_ptr()


# ---------------------------------------------------------------------------
# routing
# ---------------------------------------------------------------------------

def moe_route(logits, k: int, *, mask=None, renorm: bool = True, out: Optional[Routing] = None,
              stream=None) -> Routing:
    """The k experts of each token from its logits [T, E] (fp32 or bf16), with
    softmax weights (over the chosen experts' sum with ``renorm``), the tokens of
    each expert and the balance loss.  ``mask``: bool or uint8 [T], false leaves
    the token out.  A logit of -inf marks an expert that must not be chosen."""
    dev = logits.device
    ld = _matrix(logits, "logits")
    code = _code(logits, "logits")
    k = _count(k, "mxq_moe_route")
    where = _elsewhere(dev, stream)
    if where is not None:
        with where:
            return moe_route(logits, k, mask=mask, renorm=renorm, out=out)
    T, E = logits.shape
    mask_p = None if mask is None else _mask_pointer(mask, T, dev)
    L = lib()
    size = L.mxq_moe_route_workspace(T, E)
    ws, wp = _workspace(size, "mxq_moe_route", dev)
    if out is None:
        out = Routing(torch.empty((T, k), dtype=torch.float32, device=dev),
                      torch.empty((T, k), dtype=torch.int32, device=dev),
                      torch.empty(E, dtype=torch.int32, device=dev),
                      torch.empty((), dtype=torch.float32, device=dev),
                      torch.empty((), dtype=torch.int32, device=dev))
    else:
        for t, name, dtype, shape in zip(out, Routing._fields,
                                         (torch.float32, torch.int32, torch.int32, torch.float32, torch.int32),
                                         ((T, k), (T, k), (E,), (), ())):
            _flat(t, name, dtype, shape, dev)
    rc = L.mxq_moe_route(logits.data_ptr(), code, T, E, ld, k, mask_p, bool(renorm), out[0].data_ptr(),
                         out[1].data_ptr(), out[2].data_ptr(), out[3].data_ptr(), out[4].data_ptr(), wp, size,
                         _stream(dev.index))
    if rc != OK:
        raise MxqError(rc, "mxq_moe_route")
    return out


def moe_route_backward(logits, routing: Routing, dweights=None, dloss=None, *, mask=None,
                       renorm: bool = True, out=None, stream=None):
    """Gradient of the logits from those of the weights [T, k] and of the loss []
    (fp32; None for zero); logits, mask and renorm as in :func:`moe_route`."""
    dev = logits.device
    ld = _matrix(logits, "logits")
    code = _code(logits, "logits")
    where = _elsewhere(dev, stream)
    if where is not None:
        with where:
            return moe_route_backward(logits, routing, dweights, dloss, mask=mask, renorm=renorm, out=out)
    T, E = logits.shape
    k = routing.ids.shape[-1]
    i = _flat(routing.ids, "ids", torch.int32, (T, k), dev)
    c = _flat(routing.counts, "counts", torch.int32, (E,), dev)
    n = _flat(routing.routed, "routed", torch.int32, (), dev)
    dw = None if dweights is None else _flat(dweights, "dweights", torch.float32, (T, k), dev)
    dl = None if dloss is None else _flat(dloss, "dloss", torch.float32, (), dev)
    mask_p = None if mask is None else _mask_pointer(mask, T, dev)
    if out is None:
        out, ldd = torch.empty((T, E), dtype=logits.dtype, device=dev), E
    else:
        ldd = _matrix(out, "out", T, E, dev)
        if out.dtype != logits.dtype:
            raise ValueError("out must have the logits' type")
    rc = lib().mxq_moe_route_backward(logits.data_ptr(), code, T, E, ld, k, mask_p, bool(renorm), i, c, n, dw, dl,
                                      out.data_ptr(), ldd, _stream(dev.index))
    if rc != OK:
        raise MxqError(rc, "mxq_moe_route_backward")
    return out


_SCORES = {"sigmoid": 0, "softmax": 1}


def _score_code(scores):
    code = _SCORES.get(scores)
    if code is None:
        raise ValueError(f"scores must be one of {list(_SCORES)}")
    return code


def moe_route_groups(logits, k: int, *, bias=None, scores: str = "sigmoid", groups: int = 1, best_groups: int = 1,
                     mask=None, renorm: bool = True, scale: float = 1.0, out: Optional[Routing] = None,
                     stream=None) -> Routing:
    """The k experts of each token by their scores s ("sigmoid" or "softmax" of the logits
    [T, E]) plus ``bias`` (fp32 [E]), among the ``best_groups`` of the ``groups`` equal
    groups of experts whose two best sum highest.  Weights are ``scale`` times s of the
    chosen (over their sum with ``renorm``); tokens of each expert and the balance loss as
    in :func:`moe_route`, with s over its sum as the probabilities.  Near ties are decided
    in 64 bits."""
    dev = logits.device
    ld = _matrix(logits, "logits")
    code = _code(logits, "logits")
    what = "mxq_moe_route_groups"
    k, groups, best_groups = _count(k, what), _count(groups, what), _count(best_groups, what)
    score = _score_code(scores)
    where = _elsewhere(dev, stream)
    if where is not None:
        with where:
            return moe_route_groups(logits, k, bias=bias, scores=scores, groups=groups, best_groups=best_groups, mask=mask,
                                    renorm=renorm, scale=scale, out=out)
    T, E = logits.shape
    mask_p = None if mask is None else _mask_pointer(mask, T, dev)
    bias_p = None if bias is None else _flat(bias, "bias", torch.float32, (E,), dev)
    L = lib()
    size = L.mxq_moe_route_workspace(T, E)
    ws, wp = _workspace(size, what, dev)
    if out is None:
        out = Routing(torch.empty((T, max(k, 0)), dtype=torch.float32, device=dev),
                      torch.empty((T, max(k, 0)), dtype=torch.int32, device=dev),
                      torch.empty(E, dtype=torch.int32, device=dev),
                      torch.empty((), dtype=torch.float32, device=dev),
                      torch.empty((), dtype=torch.int32, device=dev))
    else:
        for t, name, dtype, shape in zip(out, Routing._fields,
                                         (torch.float32, torch.int32, torch.int32, torch.float32, torch.int32),
                                         ((T, k), (T, k), (E,), (), ())):
            _flat(t, name, dtype, shape, dev)
    rc = L.mxq_moe_route_groups(logits.data_ptr(), code, T, E, ld, k, bias_p, score, groups, best_groups, mask_p, bool(renorm),
                                scale, out[0].data_ptr(), out[1].data_ptr(), out[2].data_ptr(), out[3].data_ptr(),
                                out[4].data_ptr(), wp, size, _stream(dev.index))
    if rc != OK:
        raise MxqError(rc, what)
    return out


def moe_route_groups_backward(logits, routing: Routing, dweights=None, dloss=None, *, scores: str = "sigmoid", mask=None,
                              renorm: bool = True, scale: float = 1.0, out=None, stream=None):
    """Gradient of the logits of :func:`moe_route_groups` from those of the weights [T, k]
    and of the loss [] (fp32; None for zero), the choice held fixed; scores, mask, renorm
    and scale as there."""
    dev = logits.device
    ld = _matrix(logits, "logits")
    code = _code(logits, "logits")
    score = _score_code(scores)
    where = _elsewhere(dev, stream)
    if where is not None:
        with where:
            return moe_route_groups_backward(logits, routing, dweights, dloss, scores=scores, mask=mask, renorm=renorm,
                                             scale=scale, out=out)
    T, E = logits.shape
    k = routing.ids.shape[-1]
    i = _flat(routing.ids, "ids", torch.int32, (T, k), dev)
    c = _flat(routing.counts, "counts", torch.int32, (E,), dev)
    n = _flat(routing.routed, "routed", torch.int32, (), dev)
    dw = None if dweights is None else _flat(dweights, "dweights", torch.float32, (T, k), dev)
    dl = None if dloss is None else _flat(dloss, "dloss", torch.float32, (), dev)
    mask_p = None if mask is None else _mask_pointer(mask, T, dev)
    if out is None:
        out, ldd = torch.empty((T, E), dtype=logits.dtype, device=dev), E
    else:
        ldd = _matrix(out, "out", T, E, dev)
        if out.dtype != logits.dtype:
            raise ValueError("out must have the logits' type")
    rc = lib().mxq_moe_route_groups_backward(logits.data_ptr(), code, T, E, ld, k, score, mask_p, bool(renorm), scale, i, c, n,
                                             dw, dl, out.data_ptr(), ldd, _stream(dev.index))
    if rc != OK:
        raise MxqError(rc, "mxq_moe_route_groups_backward")
    return out


# ---------------------------------------------------------------------------
# exchange
# ---------------------------------------------------------------------------

def moe_rows(tokens: int, k: int, experts: int) -> int:
    """Rows that hold every routing of these sizes in groups of whole 128 rows."""
    what = "mxq_moe_rows"
    m = lib().mxq_moe_rows(_count(tokens, what), _count(k, what), _count(experts, what))
    if m < 0:
        raise MxqError(int(m), "mxq_moe_rows")
    return int(m)


def moe_plan(ids, experts: int, *, rows: Optional[int] = None, out: Optional[MoePlan] = None,
             stream=None) -> MoePlan:
    """Expert groups of the assignments ids (int32 [T, k], -1: not routed), each
    in token order and filled up to a multiple of 128 rows.  ``rows`` (at least
    :func:`moe_rows`, a multiple of 128) sets M."""
    if ids.dim() != 2:
        raise ValueError("ids must be 2-D")
    T, k = ids.shape
    dev = ids.device
    p = _flat(ids, "ids", torch.int32, (T, k), dev)
    experts = _count(experts, "mxq_moe_plan")
    rows = None if rows is None else _count(rows, "mxq_moe_plan")
    where = _elsewhere(dev, stream)
    if where is not None:
        with where:
            return moe_plan(ids, experts, rows=rows, out=out)
    L = lib()
    size = L.mxq_moe_plan_workspace(T, k, experts)
    ws, wp = _workspace(size, "mxq_moe_plan", dev)
    if out is None:
        M = L.mxq_moe_rows(T, k, experts) if rows is None else rows
        out = MoePlan(torch.empty(experts, dtype=torch.int32, device=dev),
                      torch.empty((T, k), dtype=torch.int32, device=dev),
                      torch.empty(max(M, 0), dtype=torch.int32, device=dev))
    else:
        M = out.source.numel()
        if rows is not None and rows != M:
            raise ValueError(f"out.source must have {rows} rows")
        for t, name, shape in zip(out, MoePlan._fields, ((experts,), (T, k), (M,))):
            _flat(t, name, torch.int32, shape, dev)
    rc = L.mxq_moe_plan(p, T, k, experts, M, out[0].data_ptr(), out[1].data_ptr(), out[2].data_ptr(), wp, size,
                        _stream(dev.index))
    if rc != OK:
        raise MxqError(rc, "mxq_moe_plan")
    return out


def _plan_pointers(plan, device):
    if plan.slots.dim() != 2:
        raise ValueError("slots must be 2-D")
    T, k = plan.slots.shape
    M = plan.source.numel()
    return T, k, M, _flat(plan.slots, "slots", torch.int32, (T, k), device), \
        _flat(plan.source, "source", torch.int32, (M,), device)


def moe_dispatch(x, plan: MoePlan, *, out=None, stream=None):
    """Rows [M, D] of the expert groups from the tokens' rows x [T, D] (fp32 or
    bf16); rows without an assignment are zero."""
    dev = x.device
    code = _code(x, "x")
    T, k, M, slots, source = _plan_pointers(plan, dev)
    ldx = _matrix(x, "x", T)
    where = _elsewhere(dev, stream)
    if where is not None:
        with where:
            return moe_dispatch(x, plan, out=out)
    D = x.shape[1]
    if out is None:
        out, ldr = torch.empty((M, D), dtype=x.dtype, device=dev), max(D, 1)
    else:
        ldr = _matrix(out, "out", M, D, dev)
        if out.dtype != x.dtype:
            raise ValueError("out must have x's type")
    rc = lib().mxq_moe_dispatch(x.data_ptr(), code, T, D, ldx, k, slots, source, M, out.data_ptr(), ldr,
                                _stream(dev.index))
    if rc != OK:
        raise MxqError(rc, "mxq_moe_dispatch")
    return out


def moe_combine(rows, plan: MoePlan, weights=None, *, out=None, stream=None):
    """Each token's sum over its experts of weight times row: y [T, D] from rows
    [M, D] and weights fp32 [T, k].  Without weights the plain sum, which is the
    gradient of :func:`moe_dispatch`."""
    dev = rows.device
    code = _code(rows, "rows")
    T, k, M, slots, _ = _plan_pointers(plan, dev)
    ldr = _matrix(rows, "rows", M)
    w = None if weights is None else _flat(weights, "weights", torch.float32, (T, k), dev)
    where = _elsewhere(dev, stream)
    if where is not None:
        with where:
            return moe_combine(rows, plan, weights, out=out)
    D = rows.shape[1]
    if out is None:
        out, ldy = torch.empty((T, D), dtype=rows.dtype, device=dev), max(D, 1)
    else:
        ldy = _matrix(out, "out", T, D, dev)
        if out.dtype != rows.dtype:
            raise ValueError("out must have the rows' type")
    rc = lib().mxq_moe_combine(rows.data_ptr(), code, M, D, ldr, T, k, slots, w, out.data_ptr(), ldy,
                               _stream(dev.index))
    if rc != OK:
        raise MxqError(rc, "mxq_moe_combine")
    return out


def moe_combine_backward(dy, rows, plan: MoePlan, weights, *, out=None, stream=None):
    """Gradients (drows [M, D], dweights fp32 [T, k]) of :func:`moe_combine` from
    dy [T, D]."""
    dev = rows.device
    code = _code(rows, "rows")
    T, k, M, slots, source = _plan_pointers(plan, dev)
    ldr = _matrix(rows, "rows", M)
    D = rows.shape[1]
    ldy = _matrix(dy, "dy", T, D, dev)
    if dy.dtype != rows.dtype:
        raise ValueError("dy must have the rows' type")
    w = _flat(weights, "weights", torch.float32, (T, k), dev)
    where = _elsewhere(dev, stream)
    if where is not None:
        with where:
            return moe_combine_backward(dy, rows, plan, weights, out=out)
    if out is None:
        drows, ldd = torch.empty((M, D), dtype=rows.dtype, device=dev), max(D, 1)
        dweights = torch.empty((T, k), dtype=torch.float32, device=dev)
        dw = dweights.data_ptr()
    else:
        drows, dweights = out
        ldd = _matrix(drows, "drows", M, D, dev)
        if drows.dtype != rows.dtype:
            raise ValueError("drows must have the rows' type")
        dw = _flat(dweights, "dweights", torch.float32, (T, k), dev)
    rc = lib().mxq_moe_combine_backward(dy.data_ptr(), code, T, D, ldy, rows.data_ptr(), ldr, M, k, slots, source, w,
                                        drows.data_ptr(), ldd, dw, _stream(dev.index))
    if rc != OK:
        raise MxqError(rc, "mxq_moe_combine_backward")
    return drows, dweights


# ---------------------------------------------------------------------------
# the experts' products
# ---------------------------------------------------------------------------

_ACTIVATIONS = {None: 0, "relu": 1, "silu": 2, "gelu": 3}


def _activation(name):
    code = _ACTIVATIONS.get(name)
    if code is None:
        raise ValueError(f"activation must be one of {list(_ACTIVATIONS)}")
    return code


def _offs_pointer(offs, device):
    """(pointer, G) of the groups' ends."""
    if offs is None:
        return None, 0
    if offs.dim() != 1:
        raise ValueError("offs must be 1-D")
    return _flat(offs, "offs", torch.int32, offs.shape, device), offs.numel()


def _e4m3(t, name, rows=None, cols=None, device=None):
    if t.dtype != torch.uint8:
        raise ValueError(f"{name} must be uint8 E4M3 bytes")
    return _matrix(t, name, rows, cols, device)


def _scales(t, name, count, device):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (no CPU path)")
    if t.dtype != torch.uint8 or t.numel() != count or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous uint8 tensor of {count} scales on {device}")
    return t.data_ptr()


def _output(t, name, shape, dtype, device):
    """(pitch, distance of matrices) of an output of this shape, type and device."""
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or t.device != device:
        raise ValueError(f"{name} must be a {dtype} tensor {list(shape)} on {device}")
    _, _, _, ld, stride = _stacked(t, name)
    return ld, stride


def moe_linear(q, s, w, sw, offs=None, *, bias=None, activation: Optional[str] = None, residual=None,
               preactivation: bool = False, dtype=None, out=None, stream=None):
    """The experts' product act(x w^T + bias) + residual [M, N] of rows x, given as the
    cast's row-wise bytes q [M, K] and scales s, with each group's weights, the bytes w
    [G, N, K] and scales sw of their cast.  ``offs``: the groups' ends as for
    :func:`quantize_2d_dual`; without, one group and w [N, K].  Rows behind the last
    group are zero.

    ``bias`` [G, N] ([N] without offs; fp32 or bf16), ``activation`` "relu", "silu" or
    "gelu" (tanh form), ``residual`` [M, N] of the output's type (it may be ``out``).
    With ``preactivation`` also returns z = x w^T + bias.  ``dtype``: bf16 unless given,
    or fp32.  The gradient of x is the same product of the cast dz with the column-wise
    cast of the weights (q_col of [G*N, K] as [G, K, N])."""
    dev = q.device
    ldx = _e4m3(q, "q")
    M, K = q.shape
    if w.dtype != torch.uint8:
        raise ValueError("w must be uint8 E4M3 bytes")
    if w.dim() != (2 if offs is None else 3):
        raise ValueError("w must be 3-D with offs and 2-D without")
    op, G = _offs_pointer(offs, dev)
    lead = w.shape[:-2]
    if offs is not None and w.shape[0] != G:
        raise ValueError(f"w must have {G} matrices")
    N = w.shape[-2]
    first = w if offs is None else w[0] if G > 0 else w.new_empty(N, K)
    ldw = _matrix(first, "w", N, K, dev)
    stride_w = w.stride(0) if G > 1 else 0
    code = _activation(activation)
    if dtype is None:
        dtype = torch.bfloat16 if out is None else (out[0] if preactivation else out).dtype
    if dtype not in _CODES:
        raise ValueError("dtype must be float32 or bfloat16")
    sx_p = _scales(s, "s", M * K // 32, dev)
    sw_p = _scales(sw, "sw", max(G, 1) * N * K // 32, dev)
    bias_p = bias_code = 0
    if bias is not None:
        bias_code = _code(bias, "bias")
        bias_p = _flat(bias, "bias", bias.dtype, torch.Size((*lead, N)), dev)
    ldr = res_p = 0
    if residual is not None:
        if residual.dtype != dtype:
            raise ValueError("residual must have the output's type")
        ldr, res_p = _matrix(residual, "residual", M, N, dev), residual.data_ptr()
    where = _elsewhere(dev, stream)
    if where is not None:
        with where:
            return moe_linear(q, s, w, sw, offs, bias=bias, activation=activation, residual=residual,
                              preactivation=preactivation, dtype=dtype, out=out)
    if out is None:
        y = torch.empty((M, N), dtype=dtype, device=dev)
        z = torch.empty((M, N), dtype=dtype, device=dev) if preactivation else None
        ldy = ldz = max(N, 1)
    else:
        y, z = out if preactivation else (out, None)
        ldy = _output(y, "out", (M, N), dtype, dev)[0]
        ldz = 0 if z is None else _output(z, "z", (M, N), dtype, dev)[0]
    rc = lib().mxq_moe_linear(q.data_ptr(), ldx, sx_p, w.data_ptr(), ldw, stride_w, sw_p, op, G, M, N, K, bias_p, bias_code,
                              code, res_p, ldr, _CODES[dtype], y.data_ptr(), ldy, None if z is None else z.data_ptr(), ldz,
                              _stream(dev.index))
    if rc != OK:
        raise MxqError(rc, "mxq_moe_linear")
    return (y, z) if preactivation else y


def moe_linear_backward(dy, z=None, offs=None, *, activation: Optional[str] = None, out=None, stream=None):
    """Gradients (dz [M, N], dbias fp32 [G, N], or [N] without offs) of what
    :func:`moe_linear` adds to the product: dz = dy act'(z) with the pre-activation z,
    zero behind the last group, and its sum over each group without the rows behind the
    last one.  Without an activation dz is dy itself, with those rows as they are, unless
    ``out`` has another tensor for it.  The residual's gradient is dy."""
    dev = dy.device
    dtype_code = _code(dy, "dy")
    ld = _matrix(dy, "dy")
    M, N = dy.shape
    code = _activation(activation)
    op, G = _offs_pointer(offs, dev)
    ldz = 0
    if code:
        if z is None:
            raise ValueError("z is needed with an activation")
        if z.dtype != dy.dtype:
            raise ValueError("z must have dy's type")
        ldz = _matrix(z, "z", M, N, dev)
    where = _elsewhere(dev, stream)
    if where is not None:
        with where:
            return moe_linear_backward(dy, z, offs, activation=activation, out=out)
    L = lib()
    size = L.mxq_moe_linear_backward_workspace(M, N)
    ws, wp = _workspace(size, "mxq_moe_linear_backward", dev)
    shape = (N,) if offs is None else (G, N)
    if out is None:
        dz = torch.empty((M, N), dtype=dy.dtype, device=dev) if code else dy
        dbias = torch.empty(shape, dtype=torch.float32, device=dev)
    else:
        dz, dbias = out
    ld_dz = _output(dz, "dz", (M, N), dy.dtype, dev)[0]
    dz_p = dz.data_ptr() if code or dz is not dy else None
    db = _flat(dbias, "dbias", torch.float32, torch.Size(shape), dev)
    rc = L.mxq_moe_linear_backward(dy.data_ptr(), dtype_code, ld, z.data_ptr() if code else None, ldz, code, op, G, M, N,
                                   dz_p, ld_dz, db, wp, size, _stream(dev.index))
    if rc != OK:
        raise MxqError(rc, "mxq_moe_linear_backward")
    return dz, dbias


def moe_weight_gradient(a, sa, b, sb, offs=None, *, dtype=None, out=None, accumulate: bool = False, stream=None):
    """The weights' gradient [G, N, K] of :func:`moe_linear`: for each group the product
    dz^T x over its rows, from the column-wise bytes and scales of the cast dz (a [N, M],
    sa) and of the cast x (b [K, M], sb), both with these ``offs``; [N, K] without.  fp32
    unless ``dtype`` says bf16.  With ``accumulate`` it is added to ``out``, where fp32
    numbers below 2^-126 count as 0."""
    dev = a.device
    lda = _e4m3(a, "a")
    N, M = a.shape
    ldb = _e4m3(b, "b", None, M, dev)
    K = b.shape[0]
    op, G = _offs_pointer(offs, dev)
    sa_p, sb_p = _scales(sa, "sa", N * M // 32, dev), _scales(sb, "sb", K * M // 32, dev)
    if dtype is None:
        dtype = torch.float32 if out is None else out.dtype
    if dtype not in _CODES:
        raise ValueError("dtype must be float32 or bfloat16")
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    where = _elsewhere(dev, stream)
    if where is not None:
        with where:
            return moe_weight_gradient(a, sa, b, sb, offs, dtype=dtype, out=out, accumulate=accumulate)
    shape = (N, K) if offs is None else (G, N, K)
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=dev)
    ldd, stride_d = _output(out, "out", shape, dtype, dev)
    rc = lib().mxq_moe_weight_gradient(a.data_ptr(), lda, sa_p, b.data_ptr(), ldb, sb_p, op, G, M, N, K, bool(accumulate),
                                       _CODES[dtype], out.data_ptr(), ldd, stride_d, _stream(dev.index))
    if rc != OK:
        raise MxqError(rc, "mxq_moe_weight_gradient")
    return out


# ---------------------------------------------------------------------------
# embedding table
# ---------------------------------------------------------------------------

def _ids_pointer(ids):
    if not ids.is_cuda:
        raise ValueError("ids must be a CUDA tensor (no CPU path)")
    if ids.dtype not in (torch.int32, torch.int64) or not ids.is_contiguous():
        raise ValueError("ids must be a contiguous int32 or int64 tensor")
    return ids.data_ptr(), ids.element_size()


def embedding(ids, table, *, scale: float = 1.0, dtype=None, out=None, stream=None):
    """scale * table[ids] for a table [V, D] (fp32 or bf16) and ids of any shape:
    [*ids.shape, D] of type ``dtype`` (the table's unless given).  An id outside
    the table gives zeros and sets DEV_BADINDEX in :func:`device_status`."""
    p, ib = _ids_pointer(ids)
    dev = table.device
    if ids.device != dev:
        raise ValueError(f"ids must be on {dev}")
    code = _code(table, "table")
    ldw = _matrix(table, "table")
    where = _elsewhere(dev, stream)
    if where is not None:
        with where:
            return embedding(ids, table, scale=scale, dtype=dtype, out=out)
    V, D = table.shape
    T = ids.numel()
    if out is None:
        out = torch.empty((*ids.shape, D), dtype=table.dtype if dtype is None else dtype, device=dev)
        ldy = max(D, 1)
    else:
        if dtype is not None and out.dtype != dtype:
            raise ValueError(f"out must be {dtype}")
        if out.shape != (*ids.shape, D):
            raise ValueError(f"out must be {[*ids.shape, D]}")
        ldy = _matrix(_rows_of(out, "out", T, D), "out", T, D, dev)
    rc = lib().mxq_embedding(p, ib, T, table.data_ptr(), code, V, D, ldw, scale, out.data_ptr(), _code(out, "out"), ldy,
                             _stream(dev.index))
    if rc != OK:
        raise MxqError(rc, "mxq_embedding")
    return out


def embedding_backward(ids, dy, rows: int, *, scale: float = 1.0, padding_idx: Optional[int] = None,
                       dtype=None, out=None, stream=None):
    """Gradient [rows, D] of the table of :func:`embedding` from dy [*ids.shape, D]:
    scale times the sum of dy over the tokens of each id, in fp32 and in a fixed
    order, of type ``dtype`` (dy's unless given).  Tokens with ``padding_idx`` are
    left out."""
    p, ib = _ids_pointer(ids)
    dev = dy.device
    if ids.device != dev:
        raise ValueError(f"ids must be on {dev}")
    if tuple(dy.shape[:-1]) != tuple(ids.shape):
        raise ValueError(f"dy must be {[*ids.shape]} x D")
    code = _code(dy, "dy")
    D = dy.shape[-1]
    T = ids.numel()
    ldd = _matrix(_rows_of(dy, "dy", T, D), "dy", T, D)
    rows = _count(rows, "mxq_embedding_backward")
    if padding_idx is not None and not 0 <= padding_idx < rows:
        raise ValueError(f"padding_idx must be in [0, {rows})")
    where = _elsewhere(dev, stream)
    if where is not None:
        with where:
            return embedding_backward(ids, dy, rows, scale=scale, padding_idx=padding_idx, dtype=dtype, out=out)
    L = lib()
    size = L.mxq_embedding_backward_workspace(T, rows, D)
    ws, wp = _workspace(size, "mxq_embedding_backward", dev)
    if out is None:
        out, ldw = torch.empty((rows, D), dtype=dy.dtype if dtype is None else dtype, device=dev), max(D, 1)
    else:
        if dtype is not None and out.dtype != dtype:
            raise ValueError(f"out must be {dtype}")
        ldw = _matrix(out, "out", rows, D, dev)
    rc = L.mxq_embedding_backward(p, ib, T, dy.data_ptr(), code, D, ldd, rows, -1 if padding_idx is None else padding_idx,
                                  scale, out.data_ptr(), _code(out, "out"), ldw, wp, size, _stream(dev.index))
    if rc != OK:
        raise MxqError(rc, "mxq_embedding_backward")
    return out


# ---------------------------------------------------------------------------
# orthogonalised updates
# ---------------------------------------------------------------------------

def _stacked(t, name):
    """(batch, m, n, ld, stride) of a matrix or a stack of them, rows and matrices strided."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (no CPU path)")
    if t.dim() not in (2, 3):
        raise ValueError(f"{name} must be 2-D or 3-D")
    if t.dim() == 2:
        return 1, *t.shape, _matrix(t, name), 0
    batch, m, n = t.shape
    if t.numel() == 0:
        return batch, m, n, max(n, 1), max(m * n, 1)
    ld = _matrix(t[0], name)
    stride = t.stride(0)
    if batch > 1 and stride < (m - 1) * ld + n:
        raise ValueError(f"{name} must have matrices that do not overlap")
    return batch, m, n, ld, stride if batch > 1 else 0


def orthogonalize(g, *, steps: int = 5, coefficients=(3.4445, -4.775, 2.0315), eps: float = 1e-7,
                  scale: float = 1.0, out=None, stream=None):
    """Newton-Schulz orthogonalisation of a momentum g [m, n], or of each matrix of
    a stack [batch, m, n] (fp32 or bf16): ``steps`` times X <- (aI + bA + cA^2) X
    with A = X X^T from X = g / (|g| + eps), as the Muon optimiser does.  Returns
    scale * X in bf16."""
    code = _code(g, "g")
    batch, m, n, ld, stride = _stacked(g, "g")
    a, b, c = coefficients
    steps = _count(steps, "mxq_orthogonalize")
    dev = g.device
    where = _elsewhere(dev, stream)
    if where is not None:
        with where:
            return orthogonalize(g, steps=steps, coefficients=coefficients, eps=eps, scale=scale, out=out)
    if out is None:
        out = torch.empty(g.shape, dtype=torch.bfloat16, device=dev)
    elif out.dtype != torch.bfloat16 or out.shape != g.shape or out.device != dev:
        raise ValueError(f"out must be a bfloat16 tensor {list(g.shape)} on {dev}")
    _, _, _, ldo, stride_o = _stacked(out, "out")
    L = lib()
    size = L.mxq_orthogonalize_workspace(batch, m, n)
    ws, wp = _workspace(size, "mxq_orthogonalize", dev)
    rc = L.mxq_orthogonalize(g.data_ptr(), code, batch, m, n, ld, stride, steps, a, b, c, eps, scale, out.data_ptr(), ldo,
                             stride_o, wp, size, _stream(dev.index))
    if rc != OK:
        raise MxqError(rc, "mxq_orthogonalize")
    return out


# ---------------------------------------------------------------------------
# AdamW
# ---------------------------------------------------------------------------

_START = 128           # a tensor's moments begin at a multiple of it
_TENSORS = 512         # MXQ_ADAMW_TENSORS


def _moment_starts(sizes):
    """Where each tensor's moments begin, and the elements of all."""
    starts, total = [], 0
    for n in sizes:
        starts.append(total)
        total += -(-n // _START) * _START
    return starts, total


def adamw_moments(params, bits: int = 32) -> Moments:
    """Moments of zero for :func:`adamw_step` of these parameters, on their device: fp32, or
    with ``bits`` 8 bytes and scales of MXFP8.  Those of each tensor begin at a multiple of
    128, in the order of the list."""
    if bits not in (8, 32):
        raise ValueError("bits must be 8 or 32")
    params = list(params)
    total = _moment_starts([p.numel() for p in params])[1]
    dev = params[0].device if params else torch.device("cuda", torch.cuda.current_device())
    kind = torch.float32 if bits == 32 else torch.uint8
    m, v = (torch.zeros(total, dtype=kind, device=dev) for _ in range(2))
    if bits == 32:
        return Moments(m, v, None, None)
    return Moments(m, v, *(torch.zeros(total // 32, dtype=torch.uint8, device=dev) for _ in range(2)))


def _scalar(value, name, dtype, device):
    """(number, address) of an argument that may lie on the device."""
    if not isinstance(value, torch.Tensor):
        return value, None
    return 0, _flat(value, name, dtype, (), device)


def adamw_step(params, grads, moments: Moments, step, *, lr, betas=(0.9, 0.999), eps: float = 1e-8,
               weight_decay: float = 0.01, grad_scale=None, copies=None, seed: int = 0, stream=None):
    """One AdamW step on all tensors of ``params`` in place, with their gradients, and of
    their ``moments`` (:func:`adamw_moments`):

        m = b1 m + (1 - b1) g;  v = b2 v + (1 - b2) g^2
        p = p (1 - lr weight_decay) - lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps)

    Parameters and gradients are contiguous and fp32 or bf16, each as it is; a gradient of
    None leaves its tensor and moments.  ``copies``: bf16 tensors (or None) that the new
    parameters are also rounded to.  ``step`` t counts from 1; ``step`` (int64) and ``lr``
    (fp32) may be tensors [] on the device, read as the step runs, so that a captured step
    can be replayed.  ``grad_scale``: an fp32 tensor [] that multiplies the gradients.
    Moments in 8 bits are rounded at random by ``seed`` and the step: m and the root of v
    are right on the mean, v is 2% to 5% high, and elements far below the largest of their
    32 take smaller steps.  A list that is refused
    leaves everything as it was.  Parameters and copies count as modified in place for
    autograd; the replay of a captured step is not seen by it."""
    params, grads = list(params), list(grads)
    n = len(params)
    if len(grads) != n or (copies is not None and len(copies) != n):
        raise ValueError("params, grads and copies must be of one length")
    if n == 0:
        return
    dev = params[0].device
    sizes = [p.numel() for p in params]
    starts, total = _moment_starts(sizes)
    bits = 32 if moments.m.dtype == torch.float32 else 8
    kind = torch.float32 if bits == 32 else torch.uint8
    m, v = (_flat(t, name, kind, (total,), dev) for t, name in ((moments.m, "m"), (moments.v, "v")))
    ms = vs = None
    if bits == 8:
        if moments.m_scale is None or moments.v_scale is None:
            raise ValueError("moments in 8 bits have scales")
        ms, vs = (_flat(t, name, torch.uint8, (total // 32,), dev)
                  for t, name in ((moments.m_scale, "m_scale"), (moments.v_scale, "v_scale")))
    table, live, written = [], set(), []
    for i, (p, g) in enumerate(zip(params, grads)):  # the checks of a tensor take longer than its share of a launch
        if g is None or sizes[i] == 0:
            continue
        code, gcode = _CODES.get(p.dtype), _CODES.get(g.dtype)
        if code is None or gcode is None:
            _code(p, "params"), _code(g, "grads")
        if p.device != dev or g.device != dev:
            raise ValueError("params and grads must be CUDA tensors of one device (no CPU path)")
        if not (p.is_contiguous() and g.is_contiguous() and g.shape == p.shape):
            raise ValueError("params and grads must be contiguous and of one shape")
        at, copy = p.data_ptr(), 0
        if copies is not None and copies[i] is not None:
            copy = _flat(copies[i], "copies", torch.bfloat16, p.shape, dev)
            written.append(copies[i])
        live.add(at)
        written.append(p)
        table += (at, g.data_ptr(), copy, sizes[i], starts[i], code | gcode << 32)
    if len(live) * 6 != len(table):
        raise ValueError("params must be different tensors")
    if grad_scale is not None:
        grad_scale = _flat(grad_scale, "grad_scale", torch.float32, (), dev)
    step, step_at = _scalar(step, "step", torch.int64, dev)
    lr, lr_at = _scalar(lr, "lr", torch.float32, dev)
    step, seed = index(step), index(seed)
    if not 0 <= seed < 1 << 64:
        raise ValueError("seed must be in [0, 2^64)")
    if step_at is None and not 1 <= step <= 0x7FFFFFFF:
        raise ValueError("step must count from 1")
    b1, b2 = betas
    where = _elsewhere(dev, stream)
    L, count = lib(), len(table) // 6
    table = (ctypes.c_int64 * len(table))(*table)
    if count > _TENSORS:  # several launches: all is checked before the first
        rc = L.mxq_adamw_check(table, count, bits, m, v, ms, vs, total, step_at, lr_at, grad_scale)
        if rc != OK:
            raise MxqError(rc, "mxq_adamw")
    with where if where is not None else nullcontext():
        handle = _stream(dev.index)
        for at in range(0, count, _TENSORS):
            rc = L.mxq_adamw(ctypes.byref(table, 48 * at), min(count - at, _TENSORS), bits, m, v, ms, vs, total, step, step_at,
                             lr, lr_at, b1, b2, eps, weight_decay, grad_scale, seed, handle)
            if rc != OK:
                raise MxqError(rc, "mxq_adamw")
    # written through addresses: a backward pass of a graph that saved one of them has to see it
    torch.autograd.graph.increment_version(written)
