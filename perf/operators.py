"""Measured cases of the operators between the q|k|v stage and the o projection
of a decoder layer: rotary positions, the paged KV cache (F16, Q8_0, Q4_0) as
it is written, moved and read back, and attention over that cache for single
tokens, trees of drafted tokens and prompt chunks.

``run`` computes a case in plain torch (fp32, rounded once at the end) or, with
``own`` set, through this repository's library.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TILE = 64                                  # tokens per cache tile
TYPES = {"q4_0": 0, "q8_0": 1, "f16": 16}   # cache types as the library numbers them
DT = {"f32": torch.float32, "f16": torch.float16}

# Head layouts (heads, kv heads, head dim): the 32-layer decoder's of the
# Q4_K workload, the 22-layer decoder's of the Q4_0 workload, a 64-wide one
# with 8 kv heads, one without shared heads whose dim is no power of two, and
# one with seven heads to a kv head.
LAYOUTS = [(32, 8, 128), (32, 4, 64), (32, 8, 64), (32, 32, 80), (14, 2, 64)]


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # q rotation of one decoded token: latency
        dict(name="rope_token", op="rope", tokens=1, heads=32, dim=128, rot=128, inter=False, dtype="f32",
             scaling="bands", far=9000),
        # a long prompt, 80-wide heads of which 32 dims are rotated, far positions
        dict(name="rope_prompt", op="rope", tokens=8191, heads=32, dim=80, rot=32, inter=True, dtype="f16",
             scaling="yarn", far=1000000),
        # one token of each of 5 sequences written to a Q8_0 cache
        dict(name="cache_tokens", op="cache", type="q8_0", tokens=5, kvh=8, dim=128, rot=128, inter=False,
             dtype="f32", runs=False),
        # a prompt's K and V of one layer into a Q4_0 cache, starting inside a tile
        dict(name="cache_prompt", op="cache", type="q4_0", tokens=8185, kvh=8, dim=128, rot=128, inter=False,
             dtype="f16", runs=True),
        # drafted trees written, the accepted paths moved into place and read
        dict(name="commit_pair", op="commit", type="q8_0", batch=2, tree=16, kvh=4, dim=64, dtype="f32"),
        dict(name="commit_batch", op="commit", type="f16", batch=24, tree=61, kvh=8, dim=128, dtype="f16"),
        # single tokens: a short context (latency), a long one, a ragged batch
        dict(name="decode_short", op="attn", mode="decode", type="f16", batch=1, ctx=300, tq=1, heads=32, kvh=4,
             dim=64, page=64, dtype="f32"),
        dict(name="decode_long", op="attn", mode="decode", type="q8_0", batch=1, ctx=32000, tq=1, heads=32, kvh=8,
             dim=128, page=256, dtype="f32"),
        dict(name="decode_batch", op="attn", mode="decode", type="q4_0", batch=16, ctx=8190, tq=1, heads=32, kvh=8,
             dim=128, page=64, dtype="f16"),
        # trees of drafted tokens over ragged contexts
        dict(name="tree_batch", op="attn", mode="tree", type="q8_0", batch=4, ctx=4001, tq=29, heads=32, kvh=8,
             dim=128, page=64, dtype="f32"),
        # prompt chunks of 512: the second of a prompt in two sequences, 80-wide
        # heads; the last of an 8192-token prompt
        dict(name="chunk_pair", op="attn", mode="causal", type="f16", batch=2, ctx=600, tq=512, heads=32, kvh=32,
             dim=80, page=128, dtype="f16"),
        dict(name="chunk_last", op="attn", mode="causal", type="q8_0", batch=1, ctx=7680, tq=512, heads=32, kvh=8,
             dim=128, page=64, dtype="f16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "cache", "commit", "attn", "attn", "attn"])
    heads, kvh, dim = rng.choice(LAYOUTS)
    dtype = rng.choice(["f32", "f16"])
    kind = rng.choice(["f16", "q8_0", "q4_0"])
    if op == "rope":
        return dict(op=op, tokens=_log(rng, 1, 8191), heads=rng.choice([heads, kvh]), dim=dim,
                    rot=rng.choice([dim, dim, dim // 2, 32]), inter=rng.random() < 0.5, dtype=dtype,
                    scaling=rng.choice(["none", "linear", "ntk", "yarn", "bands"]), far=_log(rng, 10000, 1000000))
    if op == "cache":
        return dict(op=op, type=kind, tokens=_log(rng, 1, 8185), kvh=kvh if kvh < 32 else 8, dim=dim,
                    rot=rng.choice([0, dim, dim, 32]), inter=rng.random() < 0.5, dtype=dtype,
                    runs=rng.random() < 0.7)
    if op == "commit":
        return dict(op=op, type=kind, batch=_log(rng, 1, 24), tree=rng.randint(2, 61), kvh=kvh, dim=dim, dtype=dtype)
    mode = rng.choice(["decode", "decode", "tree", "causal"])
    page = rng.choice([64, 128, 256])
    if mode == "decode":
        batch = _log(rng, 1, 16)
        ctx, tq = _log(rng, 1, min(32000, 8190 * 16 // batch // (2 if kvh == 32 else 1))), 1
    elif mode == "tree":
        batch = _log(rng, 1, 8)
        ctx, tq = _log(rng, 1, 8190), rng.randint(2, 64)
    else:
        batch = _log(rng, 1, 4)
        tq = _log(rng, 17, 512 // batch)
        ctx, dtype = _log(rng, 1, 7680 // batch), "f16"
    return dict(op=op, mode=mode, type=kind, batch=batch, ctx=ctx, tq=tq, heads=heads, kvh=kvh, dim=dim, page=page,
                dtype=dtype)


# ------------------------------------------------------------------ sizes --

def _blocks(dim):
    """32-value blocks of a stored head row."""
    nb = -(-dim // 32)
    return next(n for n in (2, 3, 4, 8) if n >= nb)


def _lens(case):
    """(context length, new tokens) of each sequence: ragged, the first the longest."""
    B = case["batch"]
    ctx = [max(0, case["ctx"] - (case["ctx"] * b) // (2 * B) - (b % 3)) for b in range(B)]
    tq = [case["tq"] if case["mode"] == "decode" else max(1, case["tq"] - (case["tq"] * b) // (3 * B)) for b in range(B)]
    return ctx, tq


def _value_bytes(kind):
    return {"f16": 2.0, "q8_0": 34 / 32, "q4_0": 18 / 32}[kind]


def work(case):
    es = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "rope":
        n = case["tokens"] * case["heads"] * case["dim"]
        return {"bytes": 2 * n * es + case["tokens"] * 4, "flops": 3 * case["tokens"] * case["heads"] * case["rot"]}
    if case["op"] == "cache":
        n = 2 * case["tokens"] * case["kvh"] * case["dim"]     # written, then read back as fp16
        return {"bytes": n * (es + 2 * _value_bytes(case["type"]) + 2) + case["tokens"] * case["rot"] * 4,
                "flops": 4 * n}
    if case["op"] == "commit":
        n = 2 * case["batch"] * case["kvh"] * case["dim"]
        acc = max(1, case["tree"] // 4)
        vb = _value_bytes(case["type"])
        return {"bytes": n * (case["tree"] * (es + vb) + acc * (3 * vb + 2)), "flops": 4 * n * case["tree"]}
    ctx, tq = _lens(case)
    kv = sum(c + t for c, t in zip(ctx, tq)) * case["kvh"] * case["dim"] * 2 * _value_bytes(case["type"])
    pairs = sum(t * c + t * (t + 1) // 2 for c, t in zip(ctx, tq))
    return {"bytes": kv + 2 * sum(tq) * case["heads"] * case["dim"] * es,
            "flops": 4 * pairs * case["heads"] * case["dim"]}


# ---------------------------------------------------------- the tile layout --
# A cache buffer is uint8 [pages][kv heads][tiles of a page][codes | scales].
# Within a tile of 64 tokens the codes lie in the order the matrix cores take
# them; key = 16 mq + 4 c + mr, dim = 32 b + 8 h + j:
#   K  f16   [c][b][h][mq][mr][j] fp16
#      q8_0  [c][b / g][h][mq][mr][b % g][j] bytes q + 128, g = 2 (1 if the block count is odd)
#      q4_0  [c][b / g][h][mq][mr][b % g][j / 2] bytes, dim j even in the low nibble, g = min(blocks, 4)
#      scales fp16 [key][b]
#   V, key = 16 h + 8 s + j, dim = 16 t + m:
#      f16   [t][s][h][m][j] fp16
#      q8_0  [t][h][m][8 s + j] bytes q + 128
#      q4_0  [t / 2][h][m][8 s + j] bytes, t even in the low nibble
#      scales fp16 [b][key]

def _group(kind, nb):
    return 1 if kind == "f16" else (2 if nb % 2 == 0 else 1) if kind == "q8_0" else min(nb, 4)


def _pack_k(codes, scales, kind):
    """codes [..., 64, D] (fp16 values, or integer codes) -> uint8 [..., bytes]."""
    nb, lead = codes.shape[-1] // 32, codes.shape[:-2]
    g = _group(kind, nb)
    x = codes.reshape(*lead, 4, 4, 4, nb // g, g, 4, 8)         # mq c mr bo bi h j
    n = len(lead)
    x = x.permute(*range(n), n + 1, n + 3, n + 5, n, n + 2, n + 4, n + 6)
    if kind == "f16":
        return x.contiguous().reshape(*lead, -1).view(torch.uint8)
    x = x + (128 if kind == "q8_0" else 8)
    if kind == "q4_0":
        x = x[..., 0::2] + 16 * x[..., 1::2]
    return torch.cat([x.to(torch.uint8).reshape(*lead, -1), scales.contiguous().reshape(*lead, -1).view(torch.uint8)], -1)


def _pack_v(codes, scales, kind):
    nb, lead = codes.shape[-1] // 32, codes.shape[:-2]
    n = len(lead)
    x = codes.reshape(*lead, 4, 2, 8, 2 * nb, 16)                # h s j t m
    if kind == "f16":
        return x.permute(*range(n), n + 3, n + 1, n, n + 4, n + 2).contiguous().reshape(*lead, -1).view(torch.uint8)
    x = (x + (128 if kind == "q8_0" else 8)).permute(*range(n), n + 3, n, n + 4, n + 1, n + 2)   # t h m s j
    if kind == "q4_0":
        x = x[..., 0::2, :, :, :, :] + 16 * x[..., 1::2, :, :, :, :]
    s = scales.transpose(-1, -2).contiguous()
    return torch.cat([x.to(torch.uint8).reshape(*lead, -1), s.reshape(*lead, -1).view(torch.uint8)], -1)


def _unpack(tiles, kind, nb, is_v):
    """uint8 [..., bytes] -> (codes [..., 64, D], scales [..., 64, nb]) in fp32."""
    lead, n = tiles.shape[:-1], tiles.dim() - 1
    if kind == "f16":
        x = tiles.view(torch.float16).float()
        if is_v:
            x = x.reshape(*lead, 2 * nb, 2, 4, 16, 8).permute(*range(n), n + 2, n + 1, n + 4, n, n + 3)
        else:
            x = x.reshape(*lead, 4, nb, 4, 4, 4, 8).permute(*range(n), n + 3, n, n + 4, n + 1, n + 2, n + 5)
        return x.reshape(*lead, 64, 32 * nb), None
    cb = 64 * 32 * nb // (1 if kind == "q8_0" else 2)
    code, sc = tiles[..., :cb].to(torch.int32), tiles[..., cb:].contiguous().view(torch.float16).float()
    if is_v:
        sc = sc.reshape(*lead, nb, 64).transpose(-1, -2)
        if kind == "q4_0":
            code = torch.stack([code.reshape(*lead, nb, 4, 16, 16) & 15, code.reshape(*lead, nb, 4, 16, 16) >> 4], n + 1)
        x = code.reshape(*lead, 2 * nb, 4, 16, 16).permute(*range(n), n + 1, n + 3, n, n + 2)
    else:
        sc = sc.reshape(*lead, 64, nb)
        if kind == "q4_0":
            code = torch.stack([code & 15, code >> 4], -1)
        g = _group(kind, nb)
        x = code.reshape(*lead, 4, nb // g, 4, 4, 4, g, 8).permute(*range(n), n + 3, n, n + 4, n + 1, n + 5, n + 2, n + 6)
    return (x.reshape(*lead, 64, 32 * nb) - (128 if kind == "q8_0" else 8)).float(), sc


def _encode(x, kind):
    """x fp32 [..., D] -> (codes as integers, fp32 scale before it is stored) per
    32 values: the GGUF rule in the precision of x; f16 values pass through."""
    if kind == "f16":
        return x, None
    b = x.reshape(*x.shape[:-1], -1, 32)
    if kind == "q8_0":
        d = b.abs().amax(-1) / 127
        i = torch.where(d != 0, 1 / d, torch.zeros_like(d))[..., None]
        y = b * i
        q = torch.sign(y) * torch.floor(y.abs() + 0.5)
    else:
        at = b.abs().argmax(-1, keepdim=True)
        d = b.gather(-1, at)[..., 0] / -8
        i = torch.where(d != 0, 1 / d, torch.zeros_like(d))[..., None]
        q = torch.clamp(torch.trunc(b * i + 8.5), max=15) - 8
    return q.reshape(x.shape), d


def _stored(x, kind):
    """What the cache holds of x: fp32 / fp64 values."""
    q, d = _encode(x, kind)
    if d is None:
        return x.to(torch.float16).to(x.dtype)
    d = d.to(torch.float16).to(x.dtype)
    return (q.reshape(*d.shape, 32) * d[..., None]).reshape(x.shape)


# ----------------------------------------------------------------- prepare --

def _freqs(rot, scaling, base=10000.0):
    """Angular frequency of each pair (64 bits) and the factor on cos and sin,
    scaled for four (linear, ntk), eight (bands) or sixteen (yarn) times the trained context."""
    i = np.arange(rot // 2, dtype=np.float64)
    m = 1.0
    if scaling == "ntk":
        base *= 4.0 ** (rot / max(rot - 2, 1))
    f = base ** (-2 * i / rot)
    if scaling == "linear":
        f = f / 4
    elif scaling == "bands":
        turns = 8192 * f / (2 * math.pi)
        mix = np.clip((turns - 1) / (4 - 1), 0, 1)
        f = f / 8 * (1 - mix) + f * mix
    elif scaling == "yarn":
        def at(turns):
            return rot * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(math.floor(at(32)), 0), min(math.ceil(at(1)), rot - 1)
        ramp = np.clip((i - lo) / max(hi - lo, 1e-3), 0, 1)
        f = f / 16 * ramp + f * (1 - ramp)
        m = 0.1 * math.log(16) + 1
    return f, m


def _randn(gen, *shape):
    return torch.randn(*shape, device=DEV, generator=gen)


def _table(pos, freqs, m, out=torch.float32):
    a = pos.double()[:, None] * freqs[None, :]
    return torch.stack([m * torch.cos(a), m * torch.sin(a)], -1).to(out)


def _tree(rng, n):
    """A random tree of n drafted tokens: parents and the rows of ancestor bits."""
    par = [-1] + [int(rng.integers(max(-1, i - 8), i)) for i in range(1, n)]
    bits = []
    for i, p in enumerate(par):
        bits.append((bits[p] if p >= 0 else 0) | (1 << i))
    return par, bits


def _cache_bytes(kind, kvh, dim, pages, page):
    nb = _blocks(dim)
    return pages * kvh * (page // TILE) * (64 * 32 * nb * 2 if kind == "f16" else 64 * (32 * nb // (1 if kind == "q8_0" else 2) + 2 * nb))


def _handle(s, case, k, v, pages, page):
    """The cache as a program keeps it between calls."""
    s.update(k=k, v=v, pages=pages, page=page, handle={})


def _library_cache(s, case):
    """The library's handle on the cache, made at the first call and kept."""
    import dequant_matmul_amd as qmm
    if not s["handle"]:
        s["handle"]["c"] = qmm.KVCache(TYPES[case["type"]], case["kvh"], case["dim"], s["pages"], page_size=s["page"],
                                       k=s["k"], v=s["v"])
    return qmm, s["handle"]["c"]


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    rng = np.random.default_rng(seed)
    s = {"case": case}
    if case["op"] == "rope":
        dt, T = DT[case["dtype"]], case["tokens"]
        f, m = _freqs(case["rot"], case["scaling"])
        first = int(rng.integers(0, case["far"] - T))
        s["pos"] = torch.arange(first, first + T, dtype=torch.int32, device=DEV)
        s["freqs"], s["m"] = torch.from_numpy(f).to(DEV), m
        s["x"] = _randn(gen, T, case["heads"], case["dim"]).to(dt)
        return s
    if case["op"] in ("cache", "commit"):
        dt, page = DT[case["dtype"]], 64
        if case["op"] == "cache":
            T = case["tokens"]
            pages = -(-T // page) + 5
            if case["runs"]:        # one sequence from inside a tile, its pages shuffled
                perm = torch.from_numpy(rng.permutation(pages)).to(DEV)
                at = torch.arange(T, device=DEV) + int(rng.integers(1, 60))
                s["slots"] = (perm[at // page] * page + at % page).to(torch.int32)
            else:                   # one token of each of many sequences
                s["slots"] = torch.from_numpy(rng.permutation(pages * page)[:T].astype(np.int32)).to(DEV)
            s["read"] = s["slots"][torch.from_numpy(rng.permutation(T)).to(DEV)].contiguous()
            pos, rot = torch.from_numpy(rng.integers(0, 8192, T)).to(DEV), case["rot"]
        else:
            B, n = case["batch"], case["tree"]
            T, acc = B * n, max(1, n // 4)
            per = 2                 # pages of a sequence's window
            pages = per * B + 1
            perm = rng.permutation(pages)
            slots, src, dst, depth = [], [], [], []
            for b in range(B):
                at = int(rng.integers(0, page)) + np.arange(n)
                sl = perm[per * b + at // page] * page + at % page
                par, _ = _tree(rng, n)
                path = sorted(rng.permutation(n)[:acc].tolist())
                d = [0] * n
                for i, p in enumerate(par):
                    d[i] = d[p] + 1 if p >= 0 else 0
                slots.append(sl)
                depth.append(d)
                src.append(sl[path])
                dst.append(sl[:acc])
            s["slots"] = torch.from_numpy(np.concatenate(slots).astype(np.int32)).to(DEV)
            s["src"] = torch.from_numpy(np.stack(src).astype(np.int32)).to(DEV)
            s["dst"] = torch.from_numpy(np.stack(dst).astype(np.int32)).to(DEV)
            pos, rot = torch.from_numpy(np.concatenate(depth)).to(DEV) + 1000, case["dim"]
        f, m = _freqs(rot, "none") if rot else (np.zeros(0), 1.0)
        s["cs"] = _table(pos, torch.from_numpy(f).to(DEV), m) if rot else None
        s["kin"] = _randn(gen, T, case["kvh"], case["dim"]).to(dt)
        s["vin"] = _randn(gen, T, case["kvh"], case["dim"]).to(dt)
        nbytes = _cache_bytes(case["type"], case["kvh"], case["dim"], pages, page)
        _handle(s, case, torch.zeros(nbytes, dtype=torch.uint8, device=DEV),
                torch.zeros(nbytes, dtype=torch.uint8, device=DEV), pages, page)
        return s
    # attention: a filled cache, shuffled pages, the new tokens' rows in it too
    ctx, tq = _lens(case)
    B, page, kvh, kind = case["batch"], case["page"], case["kvh"], case["type"]
    nb = _blocks(case["dim"])
    cols = max(-(-(c + t) // page) for c, t in zip(ctx, tq))
    pages = B * cols + 3
    bufs = []
    for pack in (_pack_k, _pack_v):
        shape = (pages, kvh, page // TILE, 64)
        x = torch.zeros(*shape, 32 * nb, device=DEV, dtype=torch.float16)
        x[..., :case["dim"]] = torch.randn(*shape, case["dim"], device=DEV, generator=gen, dtype=torch.float16)
        if kind == "f16":
            bufs.append(pack(x, None, kind).reshape(-1))
        else:
            q, d = _encode(x.float(), kind)
            bufs.append(pack(q.to(torch.int16), d.to(torch.float16), kind).reshape(-1))
            del q, d
        del x
    _handle(s, case, bufs[0], bufs[1], pages, page)
    s["table"] = torch.from_numpy(rng.permutation(pages)[:B * cols].reshape(B, cols).astype(np.int32)).to(DEV)
    s["ctx"] = torch.tensor(ctx, dtype=torch.int32, device=DEV)
    starts = np.concatenate([[0], np.cumsum(tq)]).astype(np.int32)
    s["qstart"] = torch.from_numpy(starts).to(DEV)
    s["q"] = _randn(gen, int(starts[-1]), case["heads"], case["dim"]).to(DT[case["dtype"]])
    s["mask"] = None
    if case["mode"] == "tree":
        words = [w - (1 << 64) if w >= 1 << 63 else w for t in tq for w in _tree(rng, t)[1]]
        s["mask"] = torch.tensor(words, dtype=torch.int64, device=DEV)[:, None]
    s["max_q"], s["max_ctx"] = max(tq), max(c + t for c, t in zip(ctx, tq))
    return s


# --------------------------------------------------------------------- run --

def _rotate(x, cs, rot, inter):
    """x [T, H, D] in the precision of cs [T, rot / 2, 2]."""
    x = x.to(cs.dtype)
    c, s = cs[:, None, :, 0], cs[:, None, :, 1]
    r = x[..., :rot]
    a, b = (r[..., 0::2], r[..., 1::2]) if inter else (r[..., :rot // 2], r[..., rot // 2:])
    u, w = a * c - b * s, b * c + a * s
    r = torch.stack([u, w], -1).flatten(-2) if inter else torch.cat([u, w], -1)
    return torch.cat([r, x[..., rot:]], -1)


def _pad(x, dim):
    """Head rows filled up to whole blocks of 32."""
    return torch.nn.functional.pad(x, (0, -dim % 32))


def _cache_rows(s, case, wide):
    """K and V rows as the cache holds them: [T, kvh, dim] in fp32 / fp64."""
    k, v, dim = s["kin"].to(wide), s["vin"].to(wide), case["dim"]
    if s["cs"] is not None:
        k = _rotate(k, s["cs"].to(wide), 2 * s["cs"].shape[1], case.get("inter", False))
    return [_stored(_pad(x, dim), case["type"])[..., :dim] for x in (k, v)]


def _attend(s, case):
    """Attention in fp32: every sequence filled up to the longest."""
    B, kvh, dim, nb = case["batch"], case["kvh"], case["dim"], _blocks(case["dim"])
    g = case["heads"] // kvh
    ctx, tab, starts = s["ctx"].long(), s["table"].long(), s["qstart"].long()
    rows = []
    for buf, is_v in ((s["k"], False), (s["v"], True)):
        t = buf.reshape(s["pages"], kvh, s["page"] // TILE, -1)[tab]           # [B, cols, kvh, tiles, bytes]
        x, d = _unpack(t, case["type"], nb, is_v)
        if d is not None:
            x = (x.reshape(*d.shape, 32) * d[..., None]).reshape(x.shape)
        rows.append(x.permute(0, 2, 1, 3, 4, 5).reshape(B, kvh, -1, 32 * nb)[:, :, :s["max_ctx"], :dim])
    k, v = rows
    L, Q = k.shape[2], s["max_q"]
    tq = starts[1:] - starts[:-1]
    i = torch.arange(Q, device=DEV)
    at = (starts[:-1, None] + i[None, :]).clamp(max=s["q"].shape[0] - 1)       # [B, Q]
    q = s["q"].float()[at].reshape(B, Q, kvh, g, dim).permute(0, 2, 3, 1, 4).reshape(B, kvh, g * Q, dim)
    j = torch.arange(L, device=DEV)
    new = j[None, None, :] - ctx[:, None, None]                                # [B, 1, L]
    if s["mask"] is None:
        see = new <= i[None, :, None]
    else:
        bit = (s["mask"][at, 0][:, :, None] >> new.clamp(0, 63)) & 1
        see = (new < 0) | ((new < tq[:, None, None]) & (bit == 1))
    sc = torch.matmul(q, k.transpose(-1, -2)) * (1 / math.sqrt(dim))
    sc = sc.reshape(B, kvh, g, Q, L).masked_fill(~see[:, None, None], -math.inf)
    sc = torch.exp(sc - sc.amax(-1, keepdim=True))
    sc = (sc / sc.sum(-1, keepdim=True)).reshape(B, kvh, g * Q, L)
    o = torch.matmul(sc, v).reshape(B, kvh, g, Q, dim).permute(0, 3, 1, 2, 4).reshape(B, Q, kvh * g, dim)
    return o[i[None, :] < tq[:, None]].to(s["q"].dtype)


def run(s):
    case = s["case"]
    if own:
        return _run_library(s, case)
    if case["op"] == "rope":
        return _rotate(s["x"], _table(s["pos"], s["freqs"], s["m"]), case["rot"], case["inter"]).to(s["x"].dtype)
    if case["op"] == "attn":
        return _attend(s, case)
    k, v = _cache_rows(s, case, torch.float32)
    out = []
    for x in (k, v):
        store = torch.zeros(s["pages"] * s["page"], *x.shape[1:], device=DEV)
        store[s["slots"].long()] = x
        if case["op"] == "commit":
            store[s["dst"].long()] = store[s["src"].long()]
        out.append(store[(s["read"] if case["op"] == "cache" else s["dst"].reshape(-1)).long()].to(torch.float16))
    return out


def _run_library(s, case):
    if case["op"] == "rope":
        import dequant_matmul_amd as qmm
        cs = qmm.rope_angles(s["pos"], s["freqs"], s["m"])
        return qmm.rope(s["x"], cs, interleaved=case["inter"])
    qmm, cache = _library_cache(s, case)
    if case["op"] == "attn":
        ws = s.setdefault("workspace", {})
        if not ws:
            ws["b"] = qmm.attention_workspace(cache, s["q"], s["table"], max_q=s["max_q"], max_ctx=s["max_ctx"])
        return qmm.attention(cache, s["q"], s["table"], s["ctx"], qstart=s["qstart"], mask=s["mask"],
                             max_q=s["max_q"], max_ctx=s["max_ctx"], workspace=ws["b"])
    qmm.kv_append(cache, s["kin"], s["vin"], s["slots"], cs=s["cs"], interleaved=case.get("inter", False))
    if case["op"] == "commit":
        qmm.kv_move(cache, s["src"], s["dst"])
        return list(qmm.kv_read(cache, s["dst"].reshape(-1), torch.float16))
    return list(qmm.kv_read(cache, s["read"], torch.float16))


# ------------------------------------------------------------------- exact --

def _places(kind, nb, dim, is_v):
    """Where a tile holds (token, dim): the index of the code in its plane
    (fp16 values or bytes), the shift of a nibble, the fp16 index of the scale."""
    key, d = torch.arange(64, device=DEV)[:, None], torch.arange(dim, device=DEV)[None, :]
    b, shift = d // 32, 0 * (key + d)
    if is_v:
        lane, t = (key // 16) * 16 + d % 16, d // 16
        if kind == "f16":
            at = ((t * 2 + key % 16 // 8) * 64 + lane) * 8 + key % 8
        elif kind == "q8_0":
            at = (t * 64 + lane) * 16 + key % 16
        else:
            at, shift = (b * 64 + lane) * 16 + key % 16, shift + 4 * (t % 2)
        scale = b * 64 + key
    else:
        lane, c, j = (d % 32 // 8) * 16 + (key // 16) * 4 + key % 4, key // 4 % 4, d % 8
        g = _group(kind, nb)
        unit = ((c * (nb // g) + b // g) * 64 + lane) * g + b % g      # of 8 dims
        at = unit * 8 + j
        if kind == "q4_0":
            at, shift = unit * 4 + j // 2, shift + 4 * (j % 2)
        scale = key * nb + b
    return at, shift, scale + 64 * 32 * nb // (2 if kind == "q8_0" else 4)


def exact(case, seed):
    """The definitions in 64 bits, one sequence at a time."""
    s = prepare(case, seed)
    dim = case["dim"]
    if case["op"] == "rope":
        a = s["pos"].double().cpu().numpy()[:, None] * s["freqs"].cpu().numpy()[None, :]
        z = torch.polar(torch.full(a.shape, float(s["m"]), dtype=torch.float64), torch.from_numpy(a)).to(DEV)
        x, rot = s["x"].double(), case["rot"]
        half = rot // 2
        p = torch.arange(half, device=DEV)
        i0, i1 = (2 * p, 2 * p + 1) if case["inter"] else (p, p + half)
        y = torch.complex(x[..., i0], x[..., i1]) * z[:, None, :]
        out = x.clone()
        out[..., i0], out[..., i1] = y.real, y.imag
        return out
    if case["op"] in ("cache", "commit"):
        out = []
        for x, turned in ((s["kin"].double(), True), (s["vin"].double(), False)):
            if turned and s["cs"] is not None:
                n = s["cs"].shape[1]
                p = torch.arange(n, device=DEV)
                i0, i1 = (2 * p, 2 * p + 1) if case.get("inter", False) else (p, p + n)
                y = torch.complex(x[..., i0], x[..., i1]) * torch.view_as_complex(s["cs"].double())[:, None, :]
                x[..., i0], x[..., i1] = y.real, y.imag
            rows = []
            for b in range(0, dim, 32):
                w = x[..., b:b + 32]
                big = w.abs().max(-1).values
                if case["type"] == "f16":
                    rows.append(w.half().double())
                elif case["type"] == "q8_0":
                    d = big / 127
                    r = w / torch.where(d > 0, d, 1.0)[..., None]
                    rows.append(torch.sign(r) * torch.floor(r.abs() + 0.5) * d.half().double()[..., None])
                else:
                    first = (w.abs() == big[..., None]).int().argmax(-1, keepdim=True)
                    d = w.gather(-1, first)[..., 0] / -8
                    r = torch.where((d == 0)[..., None], 8.0, torch.clamp(torch.floor(w / torch.where(d == 0, 1.0, d)[..., None] + 8.5), max=15.0))
                    rows.append((r - 8) * d.half().double()[..., None])
            out.append(torch.cat(rows, -1))
        where = {int(t): i for i, t in enumerate(s["slots"].tolist())}
        if case["op"] == "cache":
            at = [where[t] for t in s["read"].tolist()]
        else:
            at = [where[t] for t in s["src"].reshape(-1).tolist()]
        return [x[torch.tensor(at, device=DEV)] for x in out]
    ctx, tq = _lens(case)
    kvh, nb = case["kvh"], _blocks(dim)
    g, first, out = case["heads"] // kvh, 0, []
    places = [_places(case["type"], nb, dim, is_v) for is_v in (False, True)]
    for b in range(case["batch"]):
        n, t = ctx[b] + tq[b], tq[b]
        own_pages = s["table"][b, :-(-n // s["page"])].long()
        kv = []
        for buf, (at, shift, scale) in zip((s["k"], s["v"]), places):
            raw = buf.reshape(s["pages"], kvh, s["page"] // TILE, -1)[own_pages].transpose(0, 1)
            raw = raw.reshape(kvh, raw.shape[1] * raw.shape[2], -1)
            if case["type"] == "f16":
                x = raw.view(torch.float16)[..., at].double()
            else:
                x = ((raw[..., at] >> shift) & (255 if case["type"] == "q8_0" else 15)).double()
                x = (x - (128 if case["type"] == "q8_0" else 8)) * raw.view(torch.float16)[..., scale].double()
            kv.append(x.reshape(kvh, -1, dim)[:, :n])
        see = torch.ones(t, n, dtype=torch.bool, device=DEV)
        if s["mask"] is None:
            see[:, ctx[b]:] = torch.ones(t, t, device=DEV).tril().bool()
        else:
            w = s["mask"][first:first + t, 0].tolist()
            see[:, ctx[b]:] = torch.tensor([[(x >> j) & 1 for j in range(t)] for x in w], device=DEV).bool()
        for_heads = []
        for h in range(case["heads"]):
            q = s["q"][first:first + t, h].double()
            p = (q @ kv[0][h // g].T) / math.sqrt(dim)
            p = torch.softmax(p.masked_fill(~see, -math.inf), -1)
            for_heads.append(p @ kv[1][h // g])
        out.append(torch.stack(for_heads, 1))
        first += t
    return torch.cat(out)
