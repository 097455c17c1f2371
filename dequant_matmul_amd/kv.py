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

from . import _call, _I, _I64, _P, _SZ, lib

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


def _stream(device) -> int:
    return torch._C._cuda_getCurrentRawStream(device.index)


def _rows(t, what, tokens=None, heads=None, dim=None):
    """Checks an activation tensor [tokens, heads, dim]; its dtype code."""
    code = _DTYPES.get(t.dtype)
    if code is None or not t.is_cuda or t.dim() != 3:
        raise ValueError("%s must be a float32 or float16 device tensor [tokens, heads, head_dim]" % what)
    T, H, D = t.shape
    if (tokens is not None and T != tokens) or (heads is not None and H != heads) or (dim is not None and D != dim):
        raise ValueError("%s has shape %s, expected [%s, %s, %s]" % (what, tuple(t.shape), tokens, heads, dim))
    s = t.stride()
    if (D > 1 and s[2] != 1) or (H > 1 and s[1] != D):
        raise ValueError("the heads of a token of %s must be contiguous" % what)
    return code


def _index(t, what, device, dim=1):
    if t.dtype != torch.int32 or t.device != device or t.dim() != dim or not t.is_contiguous():
        raise ValueError("%s must be a contiguous int32 tensor of %d dimension(s) on %s" % (what, dim, device))


def _angles(cs, tokens, device):
    if cs.dtype != torch.float32 or cs.device != device or not cs.is_contiguous() or cs.dim() != 3 \
            or cs.shape[0] != tokens or cs.shape[2] != 2:
        raise ValueError("cs must be a contiguous float32 tensor [tokens, pairs, 2] on %s" % device)
    return cs.shape[1]


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
    if not pos.is_cuda:
        raise ValueError("pos must be on a HIP device")
    dev = pos.device
    _index(pos, "pos", dev)
    if freqs.dtype != torch.float64 or freqs.device != dev or freqs.dim() != 1 or not freqs.is_contiguous():
        raise ValueError("freqs must be a contiguous float64 tensor [pairs] on %s" % dev)
    T, P = pos.shape[0], freqs.shape[0]
    if out is None:
        out = torch.empty((T, P, 2), dtype=torch.float32, device=dev)
    elif out.shape != (T, P, 2) or _angles(out, T, dev) != P:
        raise ValueError("out must be [tokens, pairs, 2]")
    _call(lib.qkv_rope_angles(pos.data_ptr(), T, freqs.data_ptr(), P, magnitude, out.data_ptr(), _stream(dev)),
          "qkv_rope_angles")
    return out


def rope(x, cs, interleaved=False, out=None):
    """x [tokens, heads, head_dim] with the first 2 * pairs dims of every head
    rotated by cs (rope_angles).  out may be x (in place)."""
    code = _rows(x, "x")
    T, H, D = x.shape
    pairs = _angles(cs, T, x.device)
    if out is None:
        out = torch.empty((T, H, D), dtype=x.dtype, device=x.device)
    elif _rows(out, "out", T, H, D) != code or out.device != x.device:
        raise ValueError("out must have the type and device of x")
    _call(lib.qkv_rope(code, x.data_ptr(), x.stride(0), T, H, D, cs.data_ptr(), pairs, 1 if interleaved else 0,
                       out.data_ptr(), out.stride(0), _stream(x.device)), "qkv_rope")
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
        self.struct = CacheStruct(self.k.data_ptr(), self.v.data_ptr(), pages, qtype, kv_heads, head_dim, page_size)
        self.ptr = ctypes.addressof(self.struct)


def kv_append(cache, k, v, slots, cs=None, interleaved=False):
    """Write k and v [tokens, kv_heads, head_dim] to the slots (int32; -1
    skips a token), k rotated by cs first if given."""
    T = k.shape[0]
    code = _rows(k, "k", None, cache.kv_heads, cache.head_dim)
    if _rows(v, "v", T, cache.kv_heads, cache.head_dim) != code:
        raise ValueError("k and v must have the same type")
    dev = cache.device
    if k.device != dev or v.device != dev:
        raise ValueError("k, v and the cache must be on the same device")
    _index(slots, "slots", dev)
    if slots.shape[0] != T:
        raise ValueError("slots must have one entry per token")
    pairs = _angles(cs, T, dev) if cs is not None else 0
    _call(lib.qkv_append(cache.ptr, code, k.data_ptr(), k.stride(0), v.data_ptr(), v.stride(0), T, slots.data_ptr(),
                         cs.data_ptr() if cs is not None else None, pairs, 1 if interleaved else 0, _stream(dev)),
          "qkv_append")


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
    outs = []
    for t in (k_out, v_out):
        if t is None:
            t = torch.empty(shape, dtype=dtype, device=dev)
        elif t.dtype != dtype or tuple(t.shape) != shape or not t.is_contiguous() or t.device != dev:
            raise ValueError("outputs must be contiguous %s tensors of shape %s on %s" % (dtype, shape, dev))
        outs.append(t)
    _call(lib.qkv_read(cache.ptr, code, slots.data_ptr(), n, outs[0].data_ptr(), outs[1].data_ptr(), _stream(dev)),
          "qkv_read")
    return outs[0], outs[1]


def kv_move(cache, src, dst):
    """Copy rows src -> dst (int32 [groups, n <= 64]; -1 pads): all sources of
    a group are read before its destinations are written."""
    dev = cache.device
    _index(src, "src", dev, 2)
    _index(dst, "dst", dev, 2)
    if src.shape != dst.shape:
        raise ValueError("src and dst must have the same shape")
    _call(lib.qkv_move(cache.ptr, src.data_ptr(), dst.data_ptr(), src.shape[0], src.shape[1], _stream(dev)),
          "qkv_move")


def _attn_struct(cache, q, table, ctx, qstart, mask, max_q, max_ctx):
    code = _rows(q, "q", None, None, cache.head_dim)
    dev = cache.device
    T, H, _ = q.shape
    if q.device != dev:
        raise ValueError("q and the cache must be on the same device")
    _index(table, "table", dev, 2)
    B, cols = table.shape
    if ctx is not None:
        _index(ctx, "ctx", dev)
        if ctx.shape[0] != B:
            raise ValueError("ctx must have one entry per sequence")
    if qstart is not None:
        _index(qstart, "qstart", dev)
        if qstart.shape[0] != B + 1:
            raise ValueError("qstart must have batch + 1 entries")
    words = 0
    if mask is not None:
        if mask.dtype != torch.int64 or mask.device != dev or mask.dim() != 2 or mask.shape[0] != T \
                or not mask.is_contiguous():
            raise ValueError("mask must be a contiguous int64 tensor [tokens, words] on %s" % dev)
        words = mask.shape[1]
    if max_q is None:
        max_q = T if qstart is not None or B == 0 else -(-T // B)
    if max_ctx is None:
        max_ctx = min(cols * cache.page_size, (1 << 31) - 65)
    return AttnStruct(q.data_ptr(), None, q.stride(0), 0, T, B, table.data_ptr(), cols,
                      ctx.data_ptr() if ctx is not None else None, qstart.data_ptr() if qstart is not None else None,
                      mask.data_ptr() if words else None, words, max_q, max_ctx, None, 0, H, code, 1.0, 0)


def attention_workspace(cache, q, table, max_q=None, max_ctx=None, qstart=None):
    """A workspace tensor for attention() calls of these sizes (one call at a
    time may use it)."""
    a = _attn_struct(cache, q, table, None, qstart, None, max_q, max_ctx)
    with torch.cuda.device(cache.device):
        n = lib.qkv_attn_workspace(cache.ptr, ctypes.addressof(a))
    if n < 0:
        raise ValueError("no attention of these sizes: q %s, table %s, max_q %s, max_ctx %s"
                         % (tuple(q.shape), tuple(table.shape), max_q, max_ctx))
    return torch.empty(n, dtype=torch.uint8, device=cache.device)


def attention(cache, q, table, ctx, qstart=None, mask=None, scale=None, max_q=None, max_ctx=None, out=None,
              workspace=None):
    """Attention of q [tokens, heads, head_dim] over the cache.  table int32
    [batch, columns] page ids, ctx int32 [batch] committed tokens, qstart int32
    [batch + 1] first rows of q (None: equal shares).  mask None: new tokens see
    those up to themselves; int64 [tokens, words]: bit j of a row's words lets it
    see new token j.  scale None: head_dim ** -0.5.  max_q / max_ctx bound the
    new and all tokens of a sequence (defaults: what q and the table hold)."""
    a = _attn_struct(cache, q, table, ctx, qstart, mask, max_q, max_ctx)
    if mask is not None and a.mask_words == 0:
        raise ValueError("mask must have at least one word per row")
    dev = cache.device
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=dev)
    elif _rows(out, "out", *q.shape) != a.dtype or out.device != dev:
        raise ValueError("out must have the type and device of q")
    a.out, a.out_stride = out.data_ptr(), out.stride(0)
    a.scale = scale if scale is not None else 1.0 / math.sqrt(cache.head_dim)
    if workspace is None:
        workspace = attention_workspace(cache, q, table, max_q=max_q, max_ctx=max_ctx, qstart=qstart)
    elif workspace.dtype != torch.uint8 or workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on %s" % dev)
    a.workspace, a.workspace_bytes = workspace.data_ptr(), workspace.numel()
    _call(lib.qkv_attention(cache.ptr, ctypes.addressof(a), _stream(dev)), "qkv_attention")
    return out
