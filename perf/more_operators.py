"""Measured cases of what stands around the projections of a serving step: block
tables and slot maps made from request lengths and pages given back, the norm
with the residual's addition (fp32, fp16 or Q8_0 out), products of Q8_0
activations with quantized weights, and low-rank adapters of many requests
beside the shared projections.

``run`` computes a case in plain torch (fp32, rounded once at the end) or, with
``own`` set, through this repository's library.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
DT = {"f32": torch.float32, "f16": torch.float16}
# weight types as the library numbers them: (number, elements, bytes of a block)
TYPES = {"q4_0": (0, 32, 18), "q8_0": (1, 32, 34), "q4_k": (2, 256, 144), "q6_k": (3, 256, 210),
         "q5_0": (4, 32, 22), "q5_k": (5, 256, 176)}


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # the next token of each of 7 requests: latency
        dict(name="plan_tokens", op="plan", batch=7, ctx=5000, tq=1, page=64, scarce=False),
        # a step of many requests, prompts of up to 2048 tokens, a pool that runs out near the end
        dict(name="plan_prompts", op="plan", batch=120, ctx=9000, tq=2048, page=64, scarce=True),
        # drafted trees of a batch, the pages behind the accepted paths given back
        dict(name="trim_drafts", op="trim", batch=24, held=8200, cut=61, page=64),
        # long requests of a large batch that end
        dict(name="trim_ends", op="trim", batch=1000, held=32000, cut=32000, page=64),
        # one decoded token's norm for the 8-bit products: latency
        dict(name="norm_token", op="norm", tokens=1, heads=1, dim=4096, dtype="f32", res="f32", out="q8_0", gap=0),
        # the heads of q, views of a q|k|v projection's output, normed each by itself
        dict(name="norm_heads", op="norm", tokens=2047, heads=32, dim=128, dtype="f32", res="none", out="f16", gap=2048),
        # a long prompt: branch output fp32, residual stream fp16, fp16 for the prefill products
        dict(name="norm_prompt", op="norm", tokens=8191, heads=1, dim=4096, dtype="f32", res="f16", out="f16", gap=0),
        # the q | k | v stage of one token, the mix of types of a Q4_K_M-style file
        dict(name="q8_stage", op="q8", k=4096, batch=1, probs="q4_k:4096,q4_k:1024,q6_k:1024"),
        # gate | up of a batch of 5 tokens
        dict(name="q8_batch", op="q8", k=4096, batch=5, probs="q4_k:14336,q4_k:14336"),
        # one request with an adapter on q and v: latency
        dict(name="lora_token", op="lora", batch=1, tq=1, k=4096, outs="4096,1024", rank=16, adapters=4, dtype="f32"),
        # a decode batch of requests with adapters of mixed ranks
        dict(name="lora_batch", op="lora", batch=53, tq=1, k=4096, outs="4096,1024,1024", rank=64, adapters=24,
             dtype="f32"),
        # prompts of four requests
        dict(name="lora_prompts", op="lora", batch=4, tq=2048, k=4096, outs="4096,1024,1024", rank=32, adapters=6,
             dtype="f16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "trim", "norm", "norm", "q8", "q8", "lora", "lora"])
    page = rng.choice([64, 64, 128, 256])
    if op == "plan":
        batch = _log(rng, 1, 2000)
        tq = rng.choice([1, _log(rng, 1, max(1, min(2048, 120 * 2048 // batch)))])
        return dict(op=op, batch=batch, ctx=_log(rng, 1, 9000), tq=tq, page=page, scarce=rng.random() < 0.3)
    if op == "trim":
        batch, held = _log(rng, 1, 1000), _log(rng, 64, 32000)
        return dict(op=op, batch=batch, held=held, cut=rng.choice([min(held, rng.randint(1, 64)), _log(rng, 1, held)]),
                    page=page)
    if op == "norm":
        if rng.random() < 0.35:
            heads, dim = rng.choice([(32, 128), (8, 128), (4, 64), (32, 80), (14, 64)])
            return dict(op=op, tokens=_log(rng, 1, 2047), heads=heads, dim=dim, dtype=rng.choice(["f32", "f16"]),
                        res="none", out=rng.choice(["f32", "f16"]), gap=rng.choice([0, 8 * rng.randint(1, 300)]))
        out = rng.choice(["f32", "f16", "q8_0"])
        dim = rng.choice([2048, 4096, 5632, 896, 2560, 8192, 32 * rng.randint(2, 128)])
        if out != "q8_0" and rng.random() < 0.2:
            dim = rng.randint(1, 4097)
        return dict(op=op, tokens=_log(rng, 1, 8191 * 4096 // max(dim, 4096)), heads=1, dim=dim,
                    dtype=rng.choice(["f32", "f16"]), res=rng.choice(["none", "f32", "f16"]), out=out,
                    gap=rng.choice([0, 0, 8 * rng.randint(1, 64)]))
    if op == "q8":
        k = rng.choice([2048, 4096, 4096, 5632, 14336, 256 * rng.randint(1, 40)])
        probs = ["%s:%d" % (rng.choice(sorted(TYPES)), _log(rng, 5, 2 * 14336 * 4096 // k // 3)) for _ in range(rng.randint(1, 3))]
        return dict(op=op, k=k, batch=rng.randint(1, 8), probs=",".join(probs))
    tq = rng.choice([1, 1, _log(rng, 2, 2048)])
    batch = _log(rng, 1, 64 if tq == 1 else max(1, min(32, 4 * 2048 // tq)))
    wide = 4096 if tq == 1 else 2000
    outs = ",".join(str(rng.choice([256, 1024, 2000, wide, rng.randint(3, 2000)])) for _ in range(rng.randint(1, 3)))
    return dict(op="lora", batch=batch, tq=tq, k=8 * _log(rng, 8, 512), outs=outs, rank=8 * rng.randint(1, 4 if tq > 1 else 8),
                adapters=rng.randint(1, 24), dtype=rng.choice(["f32", "f16"]))


# ------------------------------------------------------------------- sizes --

def _ragged(most, batch, b):
    """Tokens of request b: the first has the most."""
    return max(1, most - most * b // (2 * batch) - b % 3) if most > 1 else 1


def _pages(n, page):
    return -(-n // page)


def _probs(case):
    return [(p.split(":")[0], int(p.split(":")[1])) for p in case["probs"].split(",")]


def _outs(case):
    return [int(n) for n in case["outs"].split(",")]


def _row_bytes(kind, k):
    return k // TYPES[kind][1] * TYPES[kind][2]


def work(case):
    if case["op"] == "plan":
        tokens = sum(_ragged(case["tq"], case["batch"], b) for b in range(case["batch"]))
        pages = tokens // case["page"]
        return {"bytes": 4 * (4 * case["batch"] + 2 * pages + 2 * tokens), "flops": 4 * tokens}
    if case["op"] == "trim":
        pages = case["batch"] * case["cut"] // case["page"]
        return {"bytes": 4 * (2 * case["batch"] + 2 * pages), "flops": 2 * case["batch"] + pages}
    if case["op"] == "norm":
        size = {"f32": 4, "f16": 2, "q8_0": 34 / 32, "none": 0}
        n = case["tokens"] * case["heads"] * case["dim"]
        return {"bytes": n * (size[case["dtype"]] + 2 * size[case["res"]] + size[case["out"]]) + 4 * case["dim"], "flops": 5 * n}
    if case["op"] == "q8":
        k, batch = case["k"], case["batch"]
        return {"bytes": sum(n * (_row_bytes(t, k) + 4 * batch) for t, n in _probs(case)) + batch * _row_bytes("q8_0", k),
                "flops": sum(2 * n * k * batch for _, n in _probs(case))}
    k, outs, r, batch = case["k"], _outs(case), case["rank"], case["batch"]
    tokens = sum(_ragged(case["tq"], batch, b) for b in range(batch))
    used = min(batch, case["adapters"])
    return {"bytes": used * r * 2 * (len(outs) * k + sum(outs)) + tokens * (k * (4 if case["dtype"] == "f32" else 2) + 8 * sum(outs)),
            "flops": 2 * tokens * r * (len(outs) * k + sum(outs))}


# ----------------------------------------------------------------- prepare --

def _weights(gen, kind, n, k):
    """Random blocks, uint8 [n, row bytes]: codes and packed scales of any value,
    the fp16 scales those of a file's weights."""
    _, be, bb = TYPES[kind]
    w = torch.randint(0, 256, (n, k // be, bb), device=DEV, dtype=torch.uint8, generator=gen)

    def scales(at, lo, hi):
        d = torch.rand(n, k // be, 1, device=DEV, generator=gen) * (hi - lo) + lo
        w[:, :, at:at + 2] = d.half().view(torch.uint8)
    if kind == "q6_k":
        w[:, :, 192:208] = (w[:, :, 192:208] & 127) + 192          # -64 .. 63
        scales(208, 1e-4, 1e-3)
    elif kind in ("q4_k", "q5_k"):
        scales(0, 1e-4, 1e-3)
        scales(2, 1e-4, 1e-3)
    else:
        scales(0, 1e-3, 1e-2)
    return w.reshape(n, -1)


def _hidden(gen, *shape):
    """Values as of a hidden state: normal, a few channels an order larger."""
    x = torch.randn(*shape, device=DEV, generator=gen)
    big = torch.rand(shape[-1], device=DEV, generator=gen) < 0.005
    return torch.where(big, 20 * x, x)


def _tensor(v, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(v)).to(dtype).to(DEV)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    rng = np.random.default_rng(seed)
    s = {"case": case, "keep": {}}
    if case["op"] in ("plan", "trim"):
        B, page = case["batch"], case["page"]
        if case["op"] == "plan":
            have = rng.integers(0, case["ctx"] + 1, B)
            new = np.array([_ragged(case["tq"], B, b) for b in range(B)])
            if B > 3:
                new[rng.integers(0, B, B // 8)] = 0          # requests that wait
            most = have + new
            s["fresh"], s["tokens"] = _tensor(new), sum(_ragged(case["tq"], B, b) for b in range(B)) + 5
            want = int((_pages(most, page) - _pages(have, page)).sum())
            spare = max(0, want - 1 - want // 10) if case["scarce"] else want + 40
        else:
            have = np.maximum(case["held"] - rng.integers(0, case["held"] // 2 + 1, B), 1)
            spare = 50
            s["kept"] = _tensor(np.maximum(have - case["cut"], 0))
        held = _pages(have, page)
        cols = _pages(case["ctx"] + case["tq"] if case["op"] == "plan" else case["held"], page) + 1
        total = B * cols + 50
        ids = rng.permutation(total).astype(np.int32)
        table = np.full((B, cols), -1, np.int32)
        inside = np.arange(cols)[None, :] < held[:, None]
        table[inside] = ids[:held.sum()]
        s["table"], s["ctx"] = _tensor(table), _tensor(have)
        free = np.zeros(total, np.int32)
        free[:spare] = ids[held.sum():held.sum() + spare]
        s["free"], s["count"] = _tensor(free), _tensor(np.array([spare]))
        return s
    if case["op"] == "norm":
        T, H, D = case["tokens"], case["heads"], case["dim"]
        x = _hidden(gen, T, H * D + case["gap"]).to(DT[case["dtype"]])[:, :H * D]
        s["x"] = x.unflatten(1, (H, D)) if H > 1 else x
        s["res"] = None if case["res"] == "none" else (4 * _hidden(gen, T, D)).to(DT[case["res"]])
        s["w"] = 1 + 0.2 * torch.randn(D, device=DEV, generator=gen)
        return s
    if case["op"] == "q8":
        k, batch = case["k"], case["batch"]
        s["w"] = [_weights(gen, t, n, k) for t, n in _probs(case)]
        x = _hidden(gen, batch, k).reshape(batch, k // 32, 32)
        d = x.abs().amax(-1, keepdim=True) / 127
        q = torch.round(x / d).to(torch.int8)
        s["x"] = torch.cat([d.half().view(torch.uint8), q.view(torch.uint8)], -1).reshape(batch, -1)
        return s
    B, k, r, n_ad = case["batch"], case["k"], case["rank"], case["adapters"]
    lens = [_ragged(case["tq"], B, b) for b in range(B)]
    T = sum(lens)
    s["lens"] = lens
    s["qstart"] = _tensor(np.concatenate([[0], np.cumsum(lens)]))
    pick = rng.integers(0, n_ad, B)
    if B > 4:
        pick[rng.integers(0, B, B // 5)] = -1            # requests without an adapter
    s["pick"], s["adapter"] = pick.tolist(), _tensor(pick)
    ranks = np.where(rng.random(n_ad) < 0.3, np.maximum(r // 2, 1), r)
    s["ranks_host"], s["ranks"] = ranks.tolist(), _tensor(ranks)
    s["scale"] = torch.rand(n_ad, device=DEV, generator=gen) + 0.5
    s["x"] = _hidden(gen, T, k).to(DT[case["dtype"]])
    s["a"] = [(torch.randn(n_ad, r, k, device=DEV, generator=gen) / math.sqrt(k)).half() for _ in _outs(case)]
    s["b"] = [(torch.randn(n_ad, n, r, device=DEV, generator=gen) * 0.05).half() for n in _outs(case)]
    s["base"] = [torch.randn(T, n, device=DEV, generator=gen) for n in _outs(case)]
    s["y"] = [torch.empty(T, n, device=DEV) for n in _outs(case)]
    return s


# --------------------------------------------------------------------- run --

def _plan(s, page):
    """Which requests get their pages, in order of the batch, and where each row goes."""
    c, t, cols, tokens = s["ctx"].long(), s["fresh"].long(), s["table"].shape[1], s["tokens"]
    F = s["count"].long().clamp(0, s["free"].shape[0])
    end = torch.cumsum(t.clamp(min=0), 0)
    fits = (c >= 0) & (t >= 0) & (c + t <= cols * page) & (end <= tokens)
    have = (c + page - 1) // page
    need = torch.where(fits, (c + t + page - 1) // page - have, 0)
    upto = torch.cumsum(need, 0)
    ok = fits & ((need == 0) | (upto <= F))
    left = F - torch.where(ok & (need > 0), upto, 0).max()
    j = torch.arange(cols, device=DEV)[None, :] - have[:, None]
    fill = ok[:, None] & (j >= 0) & (j < need[:, None])
    at = (F - 1 - (upto - need)[:, None] - j).clamp(0, s["free"].shape[0] - 1)
    table = torch.where(fill, s["free"][at], s["table"])
    qstart = torch.cat([torch.zeros_like(end[:1]), end]).clamp(max=tokens)
    row = torch.arange(tokens, device=DEV)
    b = torch.searchsorted(qstart[1:].contiguous(), row, right=True)
    live = b < c.shape[0]
    b = b.clamp(max=c.shape[0] - 1)
    live = live & ok[b]
    pos = torch.where(live, c[b] + row - qstart[b], 0)
    pg = table[b, pos // page].long()
    slot = torch.where(live & (pg >= 0) & (pg < s["free"].shape[0]), pg * page + pos % page, -1)
    i32 = torch.int32
    return [table, qstart.to(i32), slot.to(i32), pos.to(i32), ok.to(i32), left.to(i32)]


def _trim(s, page):
    table, held, kept = s["table"], s["ctx"].long(), s["kept"].long()
    total, F = s["free"].shape[0], s["count"].long().clamp(0, s["free"].shape[0])
    last = ((held.clamp(min=0) + page - 1) // page).clamp(max=table.shape[1])
    first = (kept.clamp(min=0) + page - 1) // page
    m = (last - first).clamp(min=0)
    upto = torch.cumsum(m, 0)
    M = torch.where(F + upto[-1] <= total, upto[-1], 0)
    j = torch.arange(table.shape[1], device=DEV)[None, :]
    goes = (j >= first[:, None]) & (j < last[:, None]) & (M > 0)
    at = F + M - 1 - (upto - m)[:, None] - (j - first[:, None])
    free = torch.cat([s["free"], s["free"][:1]])                  # one more entry takes what does not go
    free[torch.where(goes, at, total)] = table
    return [free[:total], (F + M).to(torch.int32)]


def _q8_values(y):
    """Values that Q8_0 blocks of y hold."""
    v = y.reshape(*y.shape[:-1], -1, 32)
    d = v.abs().amax(-1, keepdim=True) / 127
    z = v * torch.where(d != 0, 1 / d, torch.zeros_like(d))
    q = torch.sign(z) * torch.floor(z.abs() + 0.5)
    return (q * d.half().to(y.dtype)).reshape(y.shape)


def _norm(s, case):
    x = s["x"].float()
    out = []
    if s["res"] is not None:
        x = x + s["res"].float()
        out = [x.to(s["res"].dtype)]
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-5) * s["w"]
    return [_q8_values(y).half() if case["out"] == "q8_0" else y.to(DT[case["out"]])] + out


def _decode(w, kind, k):
    """Weights of uint8 [n, row bytes] in fp32."""
    _, be, bb = TYPES[kind]
    n = w.shape[0]
    w = w.reshape(n, k // be, bb)

    def f16(at):
        return w[:, :, at:at + 2].contiguous().view(torch.float16).float()
    if kind == "q8_0":
        return (f16(0) * w[:, :, 2:].view(torch.int8).float()).reshape(n, k)
    if kind in ("q4_0", "q5_0"):
        c = w[:, :, -16:].to(torch.int16)
        q = torch.cat([c & 15, c >> 4], -1)
        if kind == "q5_0":
            bit = torch.arange(8, device=DEV, dtype=torch.int16)
            q = q + 16 * ((w[:, :, 2:6, None].to(torch.int16) >> bit) & 1).flatten(-2)
        return (f16(0) * (q - (16 if kind == "q5_0" else 8)).float()).reshape(n, k)
    if kind in ("q4_k", "q5_k"):
        p = w[:, :, 4:16].to(torch.int16)
        sc = torch.cat([p[..., :4] & 63, (p[..., 8:] & 15) | (p[..., :4] >> 6 << 4)], -1).float()
        mn = torch.cat([p[..., 4:8] & 63, (p[..., 8:] >> 4) | (p[..., 4:8] >> 6 << 4)], -1).float()
        c = w[:, :, -128:].reshape(n, k // 256, 4, 1, 32).to(torch.int16)
        q = torch.cat([c & 15, c >> 4], -2).flatten(2, 3)                            # [n, blocks, 8, 32]
        if kind == "q5_k":
            bit = torch.arange(8, device=DEV, dtype=torch.int16)[:, None]
            q = q + 16 * ((w[:, :, None, 16:48].to(torch.int16) >> bit) & 1)
        return ((f16(0) * sc)[..., None] * q.float() - (f16(2) * mn)[..., None]).reshape(n, k)
    lo = w[:, :, :128].reshape(n, k // 256, 2, 1, 64).to(torch.int16)
    hi = w[:, :, 128:192].reshape(n, k // 256, 2, 1, 32).to(torch.int16)
    shift = torch.tensor([0, 2, 4, 6], device=DEV, dtype=torch.int16)[:, None]
    q = torch.cat([lo & 15, lo >> 4], -2).reshape(n, k // 256, 2, 4, 32) + 16 * ((hi >> shift) & 3) - 32
    d = f16(208) * w[:, :, 192:208].view(torch.int8).float()
    return (d[..., None] * q.reshape(n, k // 256, 16, 16).float()).reshape(n, k)


def _q8(s, case):
    k = case["k"]
    x = _decode(s["x"], "q8_0", k)
    return [torch.matmul(x, _decode(w, t, k).T) for w, (t, _) in zip(s["w"], _probs(case))]


def _lora(s, case):
    x, out = s["x"].float(), []
    live = torch.arange(case["rank"], device=DEV)[None, :] < s["ranks"][:, None]
    for a, b, base in zip(s["a"], s["b"], s["base"]):
        if case["tq"] == 1:              # a row a request: its own matrices, gathered
            at = s["adapter"].long().clamp(min=0)
            h = torch.matmul(a[at].float(), x[:, :, None])[:, :, 0]
            h = torch.where(live[at], h, 0) * s["scale"][at][:, None]
            y = base + torch.matmul(b[at].float(), h[:, :, None])[:, :, 0]
            out.append(torch.where((s["adapter"] >= 0)[:, None], y, base))
            continue
        y, first = base.clone(), 0
        for n, at in zip(s["lens"], s["pick"]):
            if at >= 0:
                h = torch.matmul(x[first:first + n], a[at].float().T)
                h = torch.where(live[at], h, 0) * s["scale"][at]
                y[first:first + n] += torch.matmul(h, b[at].float().T)
            first += n
        out.append(y)
    return out


def run(s):
    case = s["case"]
    if own:
        return _run_library(s, case)
    if case["op"] == "plan":
        return _plan(s, case["page"])
    if case["op"] == "trim":
        return _trim(s, case["page"])
    return {"norm": _norm, "q8": _q8, "lora": _lora}[case["op"]](s, case)


def _run_library(s, case):
    import dequant_matmul_amd as qmm
    if case["op"] == "plan":
        out = qmm.kv_plan(s["table"], s["ctx"], s["fresh"], s["free"], s["count"], s["tokens"], page_size=case["page"])
        return [s["table"], *out]
    if case["op"] == "trim":
        left = qmm.kv_trim(s["table"], s["ctx"], s["kept"], s["free"], s["count"], page_size=case["page"])
        return [s["free"], left]
    if case["op"] == "norm":
        out = qmm.rms_norm(s["x"], s["w"], residual=s["res"], eps=1e-5, dtype=DT.get(case["out"]),
                           qtype=qmm.Q8_0 if case["out"] == "q8_0" else None)
        out = [out] if s["res"] is None else list(out)
        if case["out"] == "q8_0":            # the values that the blocks stand for
            out[0] = qmm.dequant_f16(out[0], qmm.Q8_0, case["tokens"], case["dim"])
        return out
    if case["op"] == "q8":
        probs = _probs(case)
        return qmm.gemv_q8_multi(s["w"], [TYPES[t][0] for t, _ in probs], [n for _, n in probs], case["k"], s["x"])
    targets = list(zip(s["a"], s["b"], s["y"], s["base"]))
    if not s["keep"]:
        s["keep"]["ws"] = qmm.lora_workspace(s["x"], targets, s["adapter"])
    qmm.lora(s["x"], targets, s["adapter"], qstart=s["qstart"], scale=s["scale"], ranks=s["ranks"],
             workspace=s["keep"]["ws"])
    return s["y"]


# ------------------------------------------------------------------- exact --

def _code(b, kind, e):
    """Weight e of each block, b: blocks' bytes as int64 [..., bytes], in 64 bits."""
    def half(at):
        return (b[..., at] | (b[..., at + 1] << 8)).to(torch.int16).view(torch.float16).double()

    def signed(v):
        return torch.where(v > 127, v - 256, v)
    if kind == "q8_0":
        return half(0) * signed(b[..., 2 + e])
    if kind in ("q4_0", "q5_0"):
        q = (b[..., (2 if kind == "q4_0" else 6) + e % 16] >> (4 * (e // 16))) & 15
        if kind == "q4_0":
            return half(0) * (q - 8)
        return half(0) * (q + 16 * ((b[..., 2 + e // 8] >> (e % 8)) & 1) - 16)
    if kind == "q6_k":
        h, g, l = e // 128, e % 128 // 32, e % 32
        q = (b[..., 64 * h + 32 * (g % 2) + l] >> (4 * (g // 2))) & 15
        q = q + 16 * ((b[..., 128 + 32 * h + l] >> (2 * g)) & 3) - 32
        return half(208) * signed(b[..., 192 + e // 16]) * q
    j, l = e // 32, e % 32
    if j < 4:
        sc, mn = b[..., 4 + j] & 63, b[..., 8 + j] & 63
    else:
        sc = (b[..., 8 + j] & 15) + 16 * (b[..., j] >> 6)
        mn = (b[..., 8 + j] >> 4) + 16 * (b[..., 4 + j] >> 6)
    q = (b[..., (16 if kind == "q4_k" else 48) + 32 * (j // 2) + l] >> (4 * (j % 2))) & 15
    if kind == "q5_k":
        q = q + 16 * ((b[..., 16 + l] >> j) & 1)
    return half(0) * sc * q - half(2) * mn


def _wide(w, kind, k):
    _, be, bb = TYPES[kind]
    b = w.reshape(w.shape[0], k // be, bb).long()
    return torch.stack([_code(b, kind, e) for e in range(be)], -1).reshape(w.shape[0], k)


def _exact_plan(s, page):
    """One request after the other."""
    table, free = s["table"].cpu().numpy().copy(), s["free"].tolist()
    ctx, fresh, tokens = s["ctx"].tolist(), s["fresh"].tolist(), s["tokens"]
    cols, F = table.shape[1], int(s["count"][0])
    slots, pos = np.full(tokens, -1, np.int32), np.zeros(tokens, np.int32)
    qstart, ok, asked, left, row = [0], [], 0, F, 0
    for b, (c, t) in enumerate(zip(ctx, fresh)):
        good = c >= 0 and t >= 0 and c + t <= cols * page and row + max(t, 0) <= tokens
        have = -(-c // page)
        need = -(-(c + t) // page) - have if good else 0
        if good and (need == 0 or asked + need <= F):
            for i in range(need):
                table[b, have + i] = free[F - 1 - asked - i]
            if need:
                left = F - asked - need
            p = np.arange(c, c + t)
            pos[row:row + t] = p
            slots[row:row + t] = table[b, p // page] * page + p % page
            ok.append(1)
        else:
            ok.append(0)
        asked += need
        row += max(t, 0)
        qstart.append(min(row, tokens))
    return [_tensor(table), _tensor(np.array(qstart)), _tensor(slots), _tensor(pos), _tensor(np.array(ok)),
            _tensor(np.array([left]))]


def _exact_trim(s, page):
    table, free = s["table"].cpu().numpy(), s["free"].cpu().numpy().copy()
    back = []
    for row, h, n in zip(table, s["ctx"].tolist(), s["kept"].tolist()):
        back.append(row[-(-n // page):min(-(-h // page), table.shape[1])])
    back = np.concatenate(back)[::-1]
    F = int(s["count"][0])
    free[F:F + len(back)] = back
    return [_tensor(free), _tensor(np.array([F + len(back)]))]


def exact(case, seed):
    """The definitions in 64 bits."""
    s = prepare(case, seed)
    if case["op"] == "plan":
        return _exact_plan(s, case["page"])
    if case["op"] == "trim":
        return _exact_trim(s, case["page"])
    if case["op"] == "norm":
        z, out = s["x"].double(), []
        if s["res"] is not None:
            z = z + s["res"].double()
            out = [z]
        size = torch.linalg.vector_norm(z, dim=-1, keepdim=True)
        y = z / torch.sqrt(size * size / case["dim"] + 1e-5) * s["w"].double()
        if case["out"] == "q8_0":
            rows = []
            for at in range(0, case["dim"], 32):
                v = y[..., at:at + 32]
                d = v.abs().max(-1, keepdim=True).values / 127
                u = v / torch.where(d > 0, d, 1.0)
                rows.append(torch.trunc(u + torch.copysign(torch.tensor(0.5, device=DEV, dtype=u.dtype), u)) * d.half().double())
            y = torch.cat(rows, -1)
        return [y] + out
    if case["op"] == "q8":
        k, out = case["k"], []
        x = _wide(s["x"], "q8_0", k)
        for w, (t, n) in zip(s["w"], _probs(case)):
            out.append(torch.cat([_wide(w[i:i + 2048], t, k) @ x.T for i in range(0, n, 2048)]).T.contiguous())
        return out
    first, out = 0, [b.double().clone() for b in s["base"]]
    for n, at in zip(s["lens"], s["pick"]):
        rows = slice(first, first + n)
        first += n
        if at < 0:
            continue
        r, scale = s["ranks_host"][at], float(s["scale"][at])
        for a, b, y in zip(s["a"], s["b"], out):
            y[rows] += scale * (s["x"][rows].double() @ a[at, :r].double().T) @ b[at, :, :r].double().T
    return out
