"""The serving step around the projections (C ABI: ``include/qst.h``): block
tables and slot maps made on the device, the norm with the residual's addition,
products of Q8_0 activations, and adapters of many requests.

    qstart, slots, pos, granted, left = qmm.kv_plan(table, ctx, fresh, free, count, tokens)
    x8, h = qmm.rms_norm(y, w, residual=h, qtype=qmm.Q8_0)   # h + y, and its norm in Q8_0 blocks
    q, k, v = qmm.gemv_q8_multi([wq, wk, wv], types, ns, 4096, x8)
    qmm.lora(x, [(a_q, b_q, q), (a_v, b_v, v)], adapter, qstart=qstart)
    qmm.kv_append(cache, ..., slots, cs=qmm.rope_angles(pos, freqs))
    left = qmm.kv_trim(table, held, kept, free, left)        # ended requests, drafts not accepted

As the rest of the binding this module only checks and marshals arguments.
"""
from __future__ import annotations

import ctypes
import functools
import struct

import torch

from . import _call, _I, _I64, _launch, _P, Q8_0, lib, row_bytes

_I32C = ctypes.c_int32
SIGNATURES = {
    "qst_plan": (_I, [_P, _P]),
    "qst_trim": (_I, [_P, _I64, _I64, _P, _P, _P, _P, _I64, _I64, _P, _P]),
    "qst_norm": (_I, [_P, _P]),
    "qst_gemv_q8": (_I, [_I, _P, _I64, _P, _I64, _P]),
    "qst_lora_workspace": (_I64, [_P]),
    "qst_lora": (_I, [_P, _P, _P]),
}
for _name, (_res, _args) in SIGNATURES.items():
    _f = getattr(lib, _name)
    _f.restype = _res
    _f.argtypes = _args


class PlanArgs(ctypes.Structure):
    """struct qst_plan_args."""
    _fields_ = [(n, _P) for n in ("table", "ctx", "fresh", "free", "count", "qstart", "slots", "pos", "granted", "left")] \
        + [(n, _I64) for n in ("batch", "columns", "pages", "page_size", "tokens")]


class NormArgs(ctypes.Structure):
    """struct qst_norm_args."""
    _fields_ = [(n, _P) for n in ("x", "residual", "sum", "weight", "out")] \
        + [(n, _I64) for n in ("x_stride", "residual_stride", "sum_stride", "out_stride", "tokens", "heads", "dim")] \
        + [("eps", ctypes.c_float), ("x_type", _I32C), ("residual_type", _I32C), ("out_type", _I32C)]


class GemvProblem(ctypes.Structure):
    """struct qst_gemv_problem."""
    _fields_ = [("w", _P), ("y", _P), ("n", _I64), ("type", _I32C), ("reserved", _I32C)]


class LoraTarget(ctypes.Structure):
    """struct qst_lora_target."""
    _fields_ = [("a", _P), ("b", _P), ("base", _P), ("y", _P), ("n", _I64)]


class LoraArgs(ctypes.Structure):
    """struct qst_lora_args."""
    _fields_ = [(n, _P) for n in ("x", "adapter", "qstart", "scale", "ranks", "workspace")] \
        + [(n, _I64) for n in ("workspace_bytes", "x_stride", "tokens", "batch", "k")] \
        + [(n, _I32C) for n in ("adapters", "rank", "dtype", "targets")]


# These calls cost the host about as much as their kernels: the structs above are
# written as bytes (a pointer that is not given is 0), one condition checks a tensor,
# and its message is only made when it fails.
def _bytes_of(struct_class):
    """The struct.Struct that writes the fields of a ctypes structure in order."""
    code = {_P: "q", _I64: "q", _I32C: "i", ctypes.c_float: "f"}
    s = struct.Struct("@" + "".join(code[t] for _, t in struct_class._fields_))
    if s.size != ctypes.sizeof(struct_class):
        raise TypeError("fields of %s leave gaps" % struct_class.__name__)
    return s


_PLAN, _NORM, _LORA = _bytes_of(PlanArgs), _bytes_of(NormArgs), _bytes_of(LoraArgs)
_PROBLEM, _TARGET = _bytes_of(GemvProblem), _bytes_of(LoraTarget)

_F32, _F16, _I32, _U8 = torch.float32, torch.float16, torch.int32, torch.uint8
_DTYPES = {_F32: 0, _F16: 1}
_OUT_Q8 = 16 + Q8_0
_row_bytes = functools.lru_cache(maxsize=4096)(row_bytes)


def _ints(t, what, device, shape):
    if t.dtype is not _I32 or t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError("%s must be a contiguous int32 tensor of shape %s on %s" % (what, shape, device))


def _tensor(t, what, device, dtype, shape):
    if t.dtype is not dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s tensor of shape %s on %s" % (what, dtype, shape, device))


def _pool(table, free, count):
    """(device, batch, columns, pages) of a table and its pool, checked."""
    dev, size = table.device, table.shape
    if not table.is_cuda or len(size) != 2 or len(free.shape) != 1:
        raise ValueError("table must be a device tensor [batch, columns] and free [pages]")
    pages = free.shape[0]
    _ints(table, "table", dev, size)
    _ints(free, "free", dev, (pages,))
    _ints(count, "count", dev, (1,))
    return dev, size[0], size[1], pages


def kv_plan(table, ctx, fresh, free, count, tokens, page_size=64, out=None):
    """Pages, slots and positions of a step's rows: (qstart [batch + 1], slots
    [tokens], pos [tokens], granted [batch], left [1]), and the new pages' ids
    written to the table.

    table int32 [batch, columns] (page ids, updated), ctx int32 [batch] tokens
    held, fresh int32 [batch] new tokens (None: one each), free int32 [pages] the
    stack of free page ids with count int32 [1] entries, all on the device.
    tokens: rows of the batch; rows of no served request get slot -1.  Requests
    are served in order while the pool lasts (granted).  out: the five outputs
    to use; its last may be count itself."""
    dev, B, cols, pages = _pool(table, free, count)
    _ints(ctx, "ctx", dev, (B,))
    if fresh is not None:
        _ints(fresh, "fresh", dev, (B,))
    if out is None:
        # pieces of one buffer, the rows' 16-byte aligned
        pad = -tokens % 4
        slots, _, pos, _, qstart, granted, left = torch.empty(
            2 * (tokens + pad + B + 1), dtype=_I32, device=dev).split_with_sizes((tokens, pad, tokens, pad, B + 1, B, 1))
        out = (qstart, slots, pos, granted, left)
    else:
        for t, n, name in zip(out, (B + 1, tokens, tokens, B, 1), ("qstart", "slots", "pos", "granted", "left")):
            _ints(t, name, dev, (n,))
        qstart, slots, pos, granted, left = out
    a = _PLAN.pack(table.data_ptr(), ctx.data_ptr(), fresh.data_ptr() if fresh is not None else 0, free.data_ptr(),
                   count.data_ptr(), qstart.data_ptr(), slots.data_ptr(), pos.data_ptr(), granted.data_ptr(),
                   left.data_ptr(), B, cols, pages, page_size, tokens)
    status = _launch(lib.qst_plan, dev, a)
    if status:
        _call(status, "qst_plan")
    return out


def kv_trim(table, held, kept, free, count, page_size=64, left=None):
    """Pages that held[b] tokens need and kept[b] do not (int32 [batch]) go back
    to the stack; returns the new count (left; may be count itself).  The table
    stays as it is."""
    dev, B, cols, pages = _pool(table, free, count)
    _ints(held, "held", dev, (B,))
    _ints(kept, "kept", dev, (B,))
    if left is None:
        left = torch.empty_like(count)
    else:
        _ints(left, "left", dev, (1,))
    status = _launch(lib.qst_trim, dev, table.data_ptr(), B, cols, held.data_ptr(), kept.data_ptr(), free.data_ptr(),
                     count.data_ptr(), pages, page_size, left.data_ptr())
    if status:
        _call(status, "qst_trim")
    return left


def _values(t, what, shape, device):
    """(type code, token stride) of a norm's tensor, checked."""
    code, stride = _DTYPES.get(t.dtype), t.stride()
    if code is None or t.shape != shape or t.device != device:
        raise ValueError("%s must be a float32 or float16 tensor of shape %s on %s" % (what, tuple(shape), device))
    if (stride[-1] != 1 and shape[-1] > 1) or (len(shape) == 3 and stride[1] != shape[2] and shape[1] > 1):
        raise ValueError("the values of a token of %s must be contiguous" % what)
    return code, stride[0]


def rms_norm(x, weight=None, residual=None, eps=1e-6, dtype=None, qtype=None, sum_out=None, out=None):
    """Norm of the rows of x [tokens, dim], or of each head of x [tokens, heads,
    dim]: s / sqrt(mean(s^2) + eps) * weight with s = x + residual.

    Returns the norm, and with a residual (norm, s): s in the residual's type,
    written to sum_out if given (x or residual itself: in place).  dtype: float32
    or float16 (default: x's); qtype Q8_0: blocks instead, uint8 [tokens, row
    bytes].  Tokens may be strided, so views of one projection output pass as
    they are."""
    dev, shape = x.device, x.shape
    if not x.is_cuda or len(shape) not in (2, 3):
        raise ValueError("x must be a device tensor [tokens, dim] or [tokens, heads, dim]")
    code, xs = _values(x, "x", shape, dev)
    T, D = shape[0], shape[-1]
    H = shape[1] if len(shape) == 3 else 1
    rcode = scode = code
    rs = ss = 0
    if residual is not None:
        rcode, rs = _values(residual, "residual", shape, dev)
        if sum_out is None:
            sum_out = torch.empty(shape, dtype=residual.dtype, device=dev)
    if sum_out is not None:
        scode, ss = _values(sum_out, "sum_out", shape, dev)
        if scode != rcode:
            raise ValueError("sum_out must have the residual's type (without one: x's)")
    if weight is not None and (weight.dtype is not _F32 or weight.shape != (D,) or weight.device != dev
                               or not weight.is_contiguous()):
        raise ValueError("weight must be a contiguous float32 tensor [%d] on %s" % (D, dev))
    if qtype is not None:
        if qtype != Q8_0 or dtype is not None or D % 32:
            raise ValueError("qtype must be Q8_0, dim a multiple of 32 and dtype None")
        shape = (T, _row_bytes(Q8_0, H * D))
        if out is None:
            out = torch.empty(shape, dtype=_U8, device=dev)
        else:
            _tensor(out, "out", dev, _U8, shape)
        ocode, os_ = _OUT_Q8, 0
    else:
        if out is None:
            out = torch.empty(shape, dtype=dtype or x.dtype, device=dev)
        ocode, os_ = _values(out, "out", shape, dev)
        if dtype is not None and out.dtype is not dtype:
            raise ValueError("out must be of type %s" % dtype)
    a = _NORM.pack(x.data_ptr(), residual.data_ptr() if residual is not None else 0,
                   sum_out.data_ptr() if sum_out is not None else 0, weight.data_ptr() if weight is not None else 0,
                   out.data_ptr(), xs, rs, ss, os_, T, H, D, eps, code, rcode, ocode)
    status = _launch(lib.qst_norm, dev, a)
    if status:
        _call(status, "qst_norm")
    return out if residual is None else (out, sum_out)


def gemv_q8_multi(ws, qtypes, ns, k, x, outs=None):
    """y_i[b, j] = sum_l W_i[j, l] x[b, l] of weights of any block types that share
    x: uint8 [B, row_bytes(Q8_0, k)] Q8_0 blocks, B <= 8.  Returns the list of fp32
    outputs [B, n_i]."""
    if not len(ws) == len(qtypes) == len(ns):
        raise ValueError("ws, qtypes and ns must have the same length")
    dev, size = x.device, x.shape
    if x.dtype is not _U8 or not x.is_cuda or len(size) != 2 or k % 32 or size[1] != _row_bytes(Q8_0, k) \
            or not x.is_contiguous():
        raise ValueError("x must be a contiguous uint8 device tensor [B, row_bytes(Q8_0, %d)] of Q8_0 blocks" % k)
    B, n_probs = size[0], len(ws)
    if outs is None:
        outs = [None] * n_probs
    if len(outs) != n_probs:
        raise ValueError("outs must have one tensor per problem")
    for w, t, n, o in zip(ws, qtypes, ns, outs):
        if w.dtype is not _U8 or w.device != dev or not w.is_contiguous() or w.numel() != n * _row_bytes(t, k):
            raise ValueError("weights must be contiguous uint8 tensors of n * row_bytes bytes on %s" % dev)
        if o is not None:
            _tensor(o, "outs", dev, _F32, (B, n))
    outs = [torch.empty((B, n), dtype=_F32, device=dev) if o is None else o for o, n in zip(outs, ns)]
    probs = b"".join([_PROBLEM.pack(w.data_ptr(), o.data_ptr(), n, t, 0) for w, t, n, o in zip(ws, qtypes, ns, outs)])
    status = _launch(lib.qst_gemv_q8, dev, n_probs, probs, k, x.data_ptr(), B)
    if status:
        _call(status, "qst_gemv_q8")
    return outs


def gemv_q8(w, qtype, n, k, x, out=None):
    """As gemv with x in Q8_0 blocks: uint8 [B, row_bytes(Q8_0, k)] -> fp32 [B, n]."""
    return gemv_q8_multi([w], [qtype], [n], k, x, outs=None if out is None else [out])[0]


def _lora(x, targets, adapter, qstart, scale, ranks, workspace):
    """(qst_lora_args, its targets) of a call as bytes, checked."""
    dev, size, stride = x.device, x.shape, x.stride()
    code = _DTYPES.get(x.dtype)
    if code is None or not x.is_cuda or len(size) != 2 or (stride[1] != 1 and size[1] > 1):
        raise ValueError("x must be a float32 or float16 device tensor [tokens, k] with contiguous rows")
    if len(adapter.shape) != 1:
        raise ValueError("adapter must have one entry per request")
    T, k = size
    B = adapter.shape[0]
    _ints(adapter, "adapter", dev, (B,))
    if qstart is not None:
        _ints(qstart, "qstart", dev, (B + 1,))
    n_ad, rank = targets[0][0].shape[:2] if targets else (0, 8)
    tab = []
    for t in targets:
        a, b, y = t[:3]
        base = t[3] if len(t) > 3 else None
        n = y.shape[-1]
        _tensor(a, "a", dev, _F16, (n_ad, rank, k))
        _tensor(b, "b", dev, _F16, (n_ad, n, rank))
        _tensor(y, "y", dev, _F32, (T, n))
        if base is not None:
            _tensor(base, "base", dev, _F32, (T, n))
        tab.append(_TARGET.pack(a.data_ptr(), b.data_ptr(), base.data_ptr() if base is not None else 0, y.data_ptr(), n))
    if scale is not None:
        _tensor(scale, "scale", dev, _F32, (n_ad,))
    if ranks is not None:
        _ints(ranks, "ranks", dev, (n_ad,))
    ws, ws_bytes = (workspace.data_ptr(), workspace.numel()) if workspace is not None else (0, 0)
    return _LORA.pack(x.data_ptr(), adapter.data_ptr(), qstart.data_ptr() if qstart is not None else 0,
                      scale.data_ptr() if scale is not None else 0, ranks.data_ptr() if ranks is not None else 0, ws,
                      ws_bytes, stride[0], T, B, k, n_ad, rank, code, len(targets)), b"".join(tab)


def _workspace(x, targets, a):
    with torch.cuda.device(x.device):
        n = lib.qst_lora_workspace(a)
    if n < 0:
        raise ValueError("no adapters of these sizes: x %s, %d targets, first a %s"
                         % (tuple(x.shape), len(targets), tuple(targets[0][0].shape) if targets else None))
    return torch.empty(n, dtype=_U8, device=x.device)


def lora_workspace(x, targets, adapter):
    """A workspace tensor for lora() calls of these sizes (one call at a time may
    use it).  Calls of fewer tokens can need more: uint8 [4 targets tokens rank
    min(64, ceil(k / 1024))] is enough for any up to these."""
    return _workspace(x, targets, _lora(x, targets, adapter, None, None, None, None)[0])


def lora(x, targets, adapter, qstart=None, scale=None, ranks=None, workspace=None):
    """Adds the requests' adapters to the outputs of projections of x [tokens, k].

    targets: (a, b, y) or (a, b, y, base) of each projection, a float16 [adapters,
    rank, k], b float16 [adapters, n, rank], y float32 [tokens, n]; base None: y
    is added to in place, else y = base + the adapters' part.  adapter int32
    [batch]: each request's, or -1; qstart int32 [batch + 1] first rows of the
    requests (None: equal shares).  scale float32 and ranks int32 [adapters]
    (None: 1, and all of rank)."""
    dev = x.device
    if workspace is None:
        workspace = _workspace(x, targets, _lora(x, targets, adapter, qstart, scale, ranks, None)[0])
    elif workspace.dtype is not _U8 or workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on %s" % dev)
    a, tab = _lora(x, targets, adapter, qstart, scale, ranks, workspace)
    status = _launch(lib.qst_lora, dev, a, tab)
    if status:
        _call(status, "qst_lora")
