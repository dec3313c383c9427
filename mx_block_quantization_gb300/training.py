"""Operators of a mixture-of-experts training step around the MXFP8 cast.

Routing with its balance loss (:func:`moe_route`), the exchange of rows with the
128-row expert groups that :func:`quantize_2d_dual` takes (:func:`moe_plan`,
:func:`moe_dispatch`, :func:`moe_combine`), the embedding table
(:func:`embedding`) and their gradients, each a call of its own.  The functions
marshal torch CUDA tensors into the C ABI of ``include/mxq.h``, which states
each operation; there is no CPU path.

Matrices may have strided rows (unit column stride).  With ``stream`` a call runs
on that stream, and the outputs and workspaces that it allocates belong to it;
it has to be a stream of the tensors' device.  Otherwise the call runs on the current
stream of that device.
"""
from __future__ import annotations

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
