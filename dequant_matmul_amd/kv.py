"""Rotary positions, the paged KV cache and attention over it (C ABI:
``include/qkv.h``).

    freqs, m = qmm.rope_freqs(128, 500000.0)                 # host, once
    cs = qmm.rope_angles(pos, freqs.cuda(), m)               # a step's tokens: every layer uses it
    cache = qmm.KVCache(qmm.Q8_0, 8, 128, pages=512)         # a layer's K and V
    q = qmm.rope(q, cs)                                      # [tokens, heads, head_dim]
    qmm.kv_append(cache, k, v, slots, cs=cs)                 # k rotated, both quantized
    out = qmm.attention(cache, q, table, ctx)                # what the o projection reads

As the rest of the binding this module only checks and marshals arguments;
activations are float32 or float16 tensors [tokens, heads, head_dim] whose
heads are contiguous (tokens may be strided, so views of one projection output
pass as they are).
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import _call, _I, _I64, _launch, _P, _SZ, lib

F16 = 16   # cache type: plain fp16 (Q8_0 and Q4_0 are the block types)

ROPE_PLAIN, ROPE_LINEAR, ROPE_NTK, ROPE_YARN, ROPE_BANDS = range(5)
_KINDS = {"linear": ROPE_LINEAR, "ntk": ROPE_NTK, "yarn": ROPE_YARN, "bands": ROPE_BANDS}

_D = ctypes.c_double
SIGNATURES = {
    "qkv_rope_freqs": (_I, [_I64, _D, _P, _P, _P, _P]),
    "qkv_rope_angles": (_I, [_P, _I64, _P, _I64, _D, _P, _P]),
    "qkv_rope": (_I, [_I, _P, _I64, _I64, _I64, _I64, _P, _I64, _I, _P, _I64, _P]),
    "qkv_page_bytes": (_SZ, [_I, _I64, _I64, _I64]),
    "qkv_append": (_I, [_P, _I, _P, _I64, _P, _I64, _I64, _P, _P, _I64, _I, _P]),
    "qkv_read": (_I, [_P, _I, _P, _I64, _P, _P, _P]),
    "qkv_move": (_I, [_P, _P, _P, _I64, _I64, _P]),
    "qkv_attn_workspace": (_I64, [_P, _P]),
    "qkv_attention": (_I, [_P, _P, _P]),
}
for _name, (_res, _args) in SIGNATURES.items():
    _f = getattr(lib, _name)
    _f.restype = _res
    _f.argtypes = _args


class RopeScaling(ctypes.Structure):
    """struct qkv_rope_scaling."""
    _fields_ = [("kind", ctypes.c_int32), ("reserved", ctypes.c_int32), ("factor", _D), ("beta_fast", _D),
                ("beta_slow", _D), ("trained", _D), ("magnitude", _D)]


class CacheStruct(ctypes.Structure):
    """struct qkv_cache."""
    _fields_ = [("k", _P), ("v", _P), ("pages", _I64), ("type", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32)]


class AttnStruct(ctypes.Structure):
    """struct qkv_attn."""
    _fields_ = [("q", _P), ("out", _P), ("q_stride", _I64), ("out_stride", _I64), ("tokens", _I64), ("batch", _I64),
                ("table", _P), ("columns", _I64), ("ctx", _P), ("qstart", _P), ("mask", _P), ("mask_words", _I64),
                ("max_q", _I64), ("max_ctx", _I64), ("workspace", _P), ("workspace_bytes", _I64),
                ("heads", ctypes.c_int32), ("dtype", ctypes.c_int32), ("scale", ctypes.c_float),
                ("reserved", ctypes.c_int32)]


_DTYPES = {torch.float32: 0, torch.float16: 1}
_F32, _I32, _I64T, _U8 = torch.float32, torch.int32, torch.int64, torch.uint8

# The checks below stand on the path of every decoded token, where a call costs
# the host about as much as its kernel: one condition each, the message only
# made when it fails.


def _rows(t, what):
    """(dtype code, tokens, heads, head_dim, token stride) of an activation
    tensor, checked."""
    shape, stride = t.shape, t.stride()
    code = _DTYPES.get(t.dtype)
    if code is None or len(shape) != 3 or not t.is_cuda:
        raise ValueError("%s must be a float32 or float16 device tensor [tokens, heads, head_dim]" % what)
    T, H, D = shape
    if (stride[2] != 1 and D > 1) or (stride[1] != D and H > 1):
        raise ValueError("the heads of a token of %s must be contiguous" % what)
    return code, T, H, D, stride[0]


def _index(t, what, device, dim=1):
    if t.dtype is not _I32 or t.device != device or t.dim() != dim or not t.is_contiguous():
        raise ValueError("%s must be a contiguous int32 tensor of %d dimension(s) on %s" % (what, dim, device))


def _angles(cs, tokens, device):
    """The pairs of a table of angles, checked."""
    shape = cs.shape
    if cs.dtype is not _F32 or len(shape) != 3 or shape[0] != tokens or shape[2] != 2 or cs.device != device \
            or not cs.is_contiguous():
        raise ValueError("cs must be a contiguous float32 tensor [%d, pairs, 2] on %s" % (tokens, device))
    return shape[1]


def rope_freqs(rot, base=10000.0, scaling=None, factor=1.0, trained=0.0, beta_fast=None, beta_slow=1.0,
               magnitude=0.0, divisors=None):
    """(freqs float64 [rot / 2] on the host, factor on cos and sin) of `rot`
    rotated dims.  scaling: None, "linear", "ntk", "yarn" (beta_fast 32) or
    "bands" (ramp over the turns, beta_fast 4); divisors: per-pair factors."""
    if scaling is not None and scaling not in _KINDS:
        raise ValueError("scaling must be None or one of %s" % ", ".join(sorted(_KINDS)))
    sc = None
    if scaling is not None or magnitude:
        fast = beta_fast if beta_fast is not None else (4.0 if scaling == "bands" else 32.0)
        sc = RopeScaling(_KINDS[scaling] if scaling else ROPE_PLAIN, 0, factor, fast, beta_slow, trained, magnitude)
    if rot < 2 or rot % 2:
        raise ValueError("rot must be even and at least 2")
    freqs, m = torch.empty(rot // 2, dtype=torch.float64), _D()
    if divisors is not None:
        divisors = torch.as_tensor(divisors, dtype=torch.float64, device="cpu").contiguous()
        if divisors.shape != freqs.shape:
            raise ValueError("divisors must have rot / 2 values")
    _call(lib.qkv_rope_freqs(rot, base, ctypes.addressof(sc) if sc else None,
                             divisors.data_ptr() if divisors is not None else None, freqs.data_ptr(),
                             ctypes.addressof(m)), "qkv_rope_freqs")
    return freqs, m.value


def rope_angles(pos, freqs, magnitude=1.0, out=None):
    """fp32 [tokens, pairs, 2]: cos and sin (times magnitude) of pos[t] *
    freqs[i].  pos int32 [tokens], freqs float64 [pairs], both on the device."""
    dev = pos.device
    _index(pos, "pos", dev)
    if not pos.is_cuda or freqs.dtype is not torch.float64 or freqs.device != dev or freqs.dim() != 1 \
            or not freqs.is_contiguous():
        raise ValueError("pos must be on a HIP device and freqs a contiguous float64 tensor [pairs] on the same")
    T, P = pos.shape[0], freqs.shape[0]
    if out is None:
        out = torch.empty((T, P, 2), dtype=_F32, device=dev)
    elif _angles(out, T, dev) != P:
        raise ValueError("out must be [tokens, pairs, 2]")
    status = _launch(lib.qkv_rope_angles, dev, pos.data_ptr(), T, freqs.data_ptr(), P, magnitude, out.data_ptr())
    if status:
        _call(status, "qkv_rope_angles")
    return out


def rope(x, cs, interleaved=False, out=None):
    """x [tokens, heads, head_dim] with the first 2 * pairs dims of every head
    rotated by cs (rope_angles).  out may be x (in place)."""
    code, T, H, D, stride = _rows(x, "x")
    dev = x.device
    pairs = _angles(cs, T, dev)
    if out is None:
        out = torch.empty_like(x) if x.is_contiguous() else torch.empty((T, H, D), dtype=x.dtype, device=dev)
        out_stride = H * D
    else:
        got = _rows(out, "out")
        out_stride = got[4]
        if got[:4] != (code, T, H, D) or out.device != dev:
            raise ValueError("out must have the type, shape and device of x")
    status = _launch(lib.qkv_rope, dev, code, x.data_ptr(), stride, T, H, D, cs.data_ptr(), pairs, 1 if interleaved else 0,
                     out.data_ptr(), out_stride)
    if status:
        _call(status, "qkv_rope")
    return out


class KVCache:
    """The K and V pages of one layer: two uint8 buffers of `pages` pages of
    page_size tokens (a power of two, 64 or more), type F16, Q8_0 or Q4_0.
    Buffers may be given (k, v); else they are allocated, uninitialized."""

    def __init__(self, qtype, kv_heads, head_dim, pages, page_size=64, device="cuda", k=None, v=None):
        self.page_bytes = lib.qkv_page_bytes(qtype, kv_heads, head_dim, page_size)
        if self.page_bytes == 0:
            raise ValueError("no cache of type %r with kv_heads=%r, head_dim=%r, page_size=%r"
                             % (qtype, kv_heads, head_dim, page_size))
        n = pages * self.page_bytes
        for t, name in ((k, "k"), (v, "v")):
            if t is not None and (t.dtype != torch.uint8 or not t.is_cuda or not t.is_contiguous() or t.numel() != n):
                raise ValueError("%s must be a contiguous uint8 device tensor of %d bytes" % (name, n))
        if k is not None and v is not None and k.device != v.device:
            raise ValueError("k and v must be on the same device")
        if k is not None or v is not None:
            device = (k if k is not None else v).device
        self.k = k if k is not None else torch.empty(n, dtype=torch.uint8, device=device)
        self.v = v if v is not None else torch.empty(n, dtype=torch.uint8, device=device)
        self.device = self.k.device
        self.type, self.kv_heads, self.head_dim = qtype, kv_heads, head_dim
        self.pages, self.page_size = pages, page_size
        self.scale = 1.0 / math.sqrt(head_dim)
        self.struct = CacheStruct(self.k.data_ptr(), self.v.data_ptr(), pages, qtype, kv_heads, head_dim, page_size)
        self.ptr = ctypes.addressof(self.struct)


def kv_append(cache, k, v, slots, cs=None, interleaved=False):
    """Write k and v [tokens, kv_heads, head_dim] to the slots (int32; -1
    skips a token), k rotated by cs first if given."""
    code, T, H, D, k_stride = _rows(k, "k")
    got = _rows(v, "v")
    dev = cache.device
    if H != cache.kv_heads or D != cache.head_dim or got[:4] != (code, T, H, D) or k.device != dev or v.device != dev:
        raise ValueError("k and v must be [tokens, %d, %d] of one type on %s" % (cache.kv_heads, cache.head_dim, dev))
    _index(slots, "slots", dev)
    if slots.shape[0] != T:
        raise ValueError("slots must have one entry per token")
    pairs = _angles(cs, T, dev) if cs is not None else 0
    status = _launch(lib.qkv_append, dev, cache.ptr, code, k.data_ptr(), k_stride, v.data_ptr(), got[4], T, slots.data_ptr(),
                     cs.data_ptr() if cs is not None else None, pairs, 1 if interleaved else 0)
    if status:
        _call(status, "qkv_append")


def kv_read(cache, slots, dtype=torch.float32, k_out=None, v_out=None):
    """(K, V) [n, kv_heads, head_dim] of the rows at the slots (zeros for a
    slot outside the cache), float32 (exact) or float16."""
    dev = cache.device
    _index(slots, "slots", dev)
    code = _DTYPES.get(dtype)
    if code is None:
        raise ValueError("dtype must be torch.float32 or torch.float16")
    n = slots.shape[0]
    shape = (n, cache.kv_heads, cache.head_dim)
    if k_out is None and v_out is None:
        k_out = torch.empty(shape, dtype=dtype, device=dev)
        v_out = torch.empty_like(k_out)
    else:
        outs = [torch.empty(shape, dtype=dtype, device=dev) if t is None else t for t in (k_out, v_out)]
        for t in outs:
            if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.device != dev:
                raise ValueError("outputs must be contiguous %s tensors of shape %s on %s" % (dtype, shape, dev))
        k_out, v_out = outs
    status = _launch(lib.qkv_read, dev, cache.ptr, code, slots.data_ptr(), n, k_out.data_ptr(), v_out.data_ptr())
    if status:
        _call(status, "qkv_read")
    return k_out, v_out


def kv_move(cache, src, dst):
    """Copy rows src -> dst (int32 [groups, n <= 64]; -1 pads): all sources of
    a group are read before its destinations are written."""
    dev = cache.device
    _index(src, "src", dev, 2)
    _index(dst, "dst", dev, 2)
    groups, n = src.shape
    if dst.shape != src.shape:
        raise ValueError("src and dst must have the same shape")
    status = _launch(lib.qkv_move, dev, cache.ptr, src.data_ptr(), dst.data_ptr(), groups, n)
    if status:
        _call(status, "qkv_move")


def _sizes(cache, q, table, ctx, qstart, mask, max_q, max_ctx):
    """The qkv_attn of a call without its output, scale and workspace."""
    code, T, H, D, stride = _rows(q, "q")
    dev = cache.device
    if D != cache.head_dim or q.device != dev:
        raise ValueError("q must be [tokens, heads, %d] on %s" % (cache.head_dim, dev))
    _index(table, "table", dev, 2)
    B, cols = table.shape
    ctx_ptr = start_ptr = mask_ptr = None
    words = 0
    if ctx is not None:
        _index(ctx, "ctx", dev)
        if ctx.shape[0] != B:
            raise ValueError("ctx must have one entry per sequence")
        ctx_ptr = ctx.data_ptr()
    if qstart is not None:
        _index(qstart, "qstart", dev)
        if qstart.shape[0] != B + 1:
            raise ValueError("qstart must have batch + 1 entries")
        start_ptr = qstart.data_ptr()
    if mask is not None:
        if mask.dtype is not _I64T or mask.device != dev or mask.dim() != 2 or mask.shape[0] != T \
                or mask.shape[1] == 0 or not mask.is_contiguous():
            raise ValueError("mask must be a contiguous int64 tensor [tokens, words] on %s" % dev)
        mask_ptr, words = mask.data_ptr(), mask.shape[1]
    if max_q is None:
        max_q = T if qstart is not None or B == 0 else -(-T // B)
    if max_ctx is None:
        max_ctx = min(cols * cache.page_size, (1 << 31) - 65)
    return AttnStruct(q.data_ptr(), None, stride, H * D, T, B, table.data_ptr(), cols, ctx_ptr, start_ptr, mask_ptr,
                      words, max_q, max_ctx, None, 0, H, code, 1.0, 0)


def attention_workspace(cache, q, table, max_q=None, max_ctx=None, qstart=None):
    """A workspace tensor for attention() calls of these sizes (one call at a
    time may use it).  Fewer sequences or rows may need more: one kept for several
    batches is the largest of theirs."""
    a = _sizes(cache, q, table, None, qstart, None, max_q, max_ctx)
    with torch.cuda.device(cache.device):
        n = lib.qkv_attn_workspace(cache.ptr, ctypes.addressof(a))
    if n < 0:
        raise ValueError("no attention of these sizes: q %s, table %s, max_q %s, max_ctx %s"
                         % (tuple(q.shape), tuple(table.shape), max_q, max_ctx))
    return torch.empty(n, dtype=_U8, device=cache.device)


def attention(cache, q, table, ctx, qstart=None, mask=None, scale=None, max_q=None, max_ctx=None, out=None,
              workspace=None):
    """Attention of q [tokens, heads, head_dim] over the cache.  table int32
    [batch, columns] page ids, ctx int32 [batch] committed tokens, qstart int32
    [batch + 1] first rows of q (None: equal shares).  mask None: new tokens see
    those up to themselves; int64 [tokens, words]: bit j of a row's words lets it
    see new token j.  scale None: head_dim ** -0.5.  max_q / max_ctx bound the
    new and all tokens of a sequence (defaults: what q and the table hold); they
    choose the kernel and its splits, so close bounds are faster.  Rows of q that
    belong to no sequence are not written."""
    a = _sizes(cache, q, table, ctx, qstart, mask, max_q, max_ctx)
    dev = cache.device
    if out is None:
        out = torch.empty_like(q) if q.is_contiguous() else torch.empty(q.shape, dtype=q.dtype, device=dev)
    else:
        got = _rows(out, "out")
        if out.shape != q.shape or got[0] != a.dtype or out.device != dev:
            raise ValueError("out must have the type, shape and device of q")
        a.out_stride = got[4]
    a.out = out.data_ptr()
    a.scale = scale if scale is not None else cache.scale
    if workspace is None:
        workspace = attention_workspace(cache, q, table, max_q=max_q, max_ctx=max_ctx, qstart=qstart)
    elif workspace.dtype is not _U8 or workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on %s" % dev)
    a.workspace, a.workspace_bytes = workspace.data_ptr(), workspace.numel()
    status = _launch(lib.qkv_attention, dev, cache.ptr, ctypes.addressof(a))
    if status:
        _call(status, "qkv_attention")
    return out
