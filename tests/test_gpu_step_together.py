"""The serving step as it is used: pages planned, norms, 8-bit products, adapters,
rotation, cache, attention and pages given back, over the steps of a batch, against
the same in 64 bits; calls captured in a graph and replayed, on other streams, and
two at once."""
import numpy as np
import pytest

import oracle
import qmm_inputs as G
import step_ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import dequant_matmul_amd as q  # noqa: E402

DEV = "cuda:0"
I32 = torch.int32


def up(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    return t if dtype is None else t.to(dtype)


class Layer:
    """An attention block of a decoder layer: 4 heads on 2 kv heads of 64, width 512."""
    H, KVH, D, W = 4, 2, 64, 512

    def __init__(self, seed, adapters=3, rank=16):
        gen = torch.Generator().manual_seed(seed)
        self.types = [G.Q4_K, G.Q4_K, G.Q6_K]
        self.ns = [self.H * self.D, self.KVH * self.D, self.KVH * self.D]
        self.host = [G.gen_weights(t, n, self.W, seed + i, d_range=(1e-5, 1e-4)) for i, (t, n) in enumerate(zip(self.types, self.ns))]
        self.w = [up(h) for h in self.host]
        self.norm = 1 + 0.2 * torch.randn(self.W, generator=gen)
        self.qnorm = 1 + 0.2 * torch.randn(self.D, generator=gen)
        self.a = [(torch.randn(adapters, rank, self.W, generator=gen) / self.W ** 0.5).half() for _ in self.ns]
        self.b = [(torch.randn(adapters, n, rank, generator=gen) * 0.1).half() for n in self.ns]
        self.freqs, self.m = q.rope_freqs(self.D, 10000.0)


def attend(rows, k, v, ctx):
    """rows [t, H, D] after ctx cached tokens, k and v [ctx + t, KVH, D], in 64 bits."""
    t, H, D = rows.shape
    g = H // k.shape[1]
    z = torch.einsum("ihd,jhd->hij", rows, k.repeat_interleave(g, 1)) / D ** 0.5
    z.masked_fill_(torch.ones(t, ctx + t, dtype=torch.bool).triu(ctx + 1), -np.inf)
    return torch.einsum("hij,jhd->ihd", z.softmax(-1), v.repeat_interleave(g, 1))


def test_steps_of_a_batch():
    """A prompt of one request beside single tokens of others, then single tokens of
    all, drafted rows of which some are taken back, one request ending and its pages
    going to another.  The cache's rows are read back, so that what the projections
    and adapters made is compared with 64 bits, and attention over them again."""
    L, page, cols, pages, B = Layer(1), 64, 6, 14, 4
    gen = torch.Generator().manual_seed(3)
    rng = np.random.default_rng(4)
    cache = q.KVCache(q.F16, L.KVH, L.D, pages, page)
    table = torch.full((B, cols), -1, dtype=I32, device=DEV)
    free, count = up(rng.permutation(pages).astype(np.int32)), up(np.array([pages], np.int32))
    ctx = np.zeros(B, np.int64)
    adapter = np.array([2, -1, 0, 2], np.int32)
    dev = [t.to(DEV) for t in (L.norm, L.qnorm)]
    ad = [(a.to(DEV), b.to(DEV)) for a, b in zip(L.a, L.b)]
    freqs = L.freqs.to(DEV)
    held_pages = lambda n: -(-n // page)  # noqa: E731
    Wq = [torch.from_numpy(oracle.dequant(t, h, n, L.W)).double() for t, h, n in zip(L.types, L.host, L.ns)]
    steps = [([130, 1, 5, 0], [0, 0, 0, 0]), ([1, 1, 1, 1], [0, 0, 0, 0]), ([3, 2, 1, 60], [2, 0, 0, 31]),
             ([1, 1, 1, 1], [0, 0, 0, 0]), ([1, 0, 1, 1], [0, 200, 0, 0]), ([2, 1, 1, 130], [0, 0, 0, 0])]
    for fresh, drop in steps:
        fresh = np.array(fresh)
        T = int(fresh.sum())
        x, h = torch.randn(T + 3, L.W, generator=gen), torch.randn(T + 3, L.W, generator=gen)
        tab0, free0, count0 = table.cpu().numpy(), free.cpu().numpy(), int(count[0])
        qstart, slots, pos, granted, count = q.kv_plan(table, up(ctx.astype(np.int32)), up(fresh.astype(np.int32)), free,
                                                       count, T + 3, page_size=page)
        want = step_ref.plan(tab0, ctx, fresh, free0, count0, T + 3, page)
        for got, w in zip((table, qstart, slots, pos, granted), want):
            assert np.array_equal(got.cpu().numpy(), w)
        assert int(count[0]) == want[5] and want[4].all()
        # the layer, up to 8 rows a product (decode), adapters and norms for all rows at once
        hidden, total = q.rms_norm(x.to(DEV), dev[0], residual=h.to(DEV), qtype=q.Q8_0)
        outs = [torch.empty(T + 3, n, device=DEV) for n in L.ns]
        for r in range(0, T + 3, 8):
            part = hidden[r:r + 8].contiguous()
            for o, y in zip(outs, q.gemv_q8_multi(L.w, L.types, L.ns, L.W, part)):
                o[r:r + 8] = y
        plain = [o.clone() for o in outs]
        values = q.dequant(hidden, q.Q8_0, T + 3, L.W)
        q.lora(values, [(a, b, o) for (a, b), o in zip(ad, outs)], up(adapter), qstart=qstart)
        assert all(torch.equal(o[T:], p[T:]) for o, p in zip(outs, plain))
        rows = q.rms_norm(outs[0].view(T + 3, L.H, L.D), dev[1])
        cs = q.rope_angles(pos, freqs, L.m)
        rows = q.rope(rows, cs)
        q.kv_append(cache, outs[1].view(-1, L.KVH, L.D), outs[2].view(-1, L.KVH, L.D), slots, cs=cs)
        out = q.attention(cache, rows, table, up(ctx.astype(np.int32)), qstart=qstart)
        # 64 bits: products and adapters of the decoded hidden rows
        v64 = values.double().cpu()
        s64, _ = step_ref.norm(x.numpy(), h.numpy(), L.norm.numpy(), 1e-6)
        assert np.abs(total.double().cpu().numpy() - s64).max() < 1e-6
        bases = [(v64 @ w.T).numpy() for w in Wq]
        starts = want[1]
        ref = step_ref.lora(v64.numpy(), adapter, starts, [(a.numpy(), b.numpy(), y) for a, b, y in zip(L.a, L.b, bases)], None, None)
        for o, (y, mag, top), w in zip(outs, ref, Wq):
            # the products' own bar of 2e-5 of their magnitude, the adapters' of a quarter of k roundings
            bar = 2e-5 * (v64.abs() @ w.abs().T).numpy() + 200 * 2.0 ** -24 * mag + 2.0 ** -21 * top
            assert np.all(np.abs(o.double().cpu().numpy() - y)[:T] <= bar[:T])
        # attention again from what the cache holds
        tb = table.cpu().numpy()
        for b in range(B):
            n, t = ctx[b] + fresh[b], fresh[b]
            if t == 0:
                continue
            p = np.arange(n)
            k, v = q.kv_read(cache, up((tb[b, p // page] * page + p % page).astype(np.int32)), torch.float32)
            y = attend(rows[starts[b]:starts[b + 1]].double().cpu(), k.double().cpu(), v.double().cpu(), int(ctx[b]))
            assert (out[starts[b]:starts[b + 1]].double().cpu() - y).abs().max() < 2e-5 * max(1.0, float(v.abs().max()))
        # drafts not taken and ended requests give their pages back
        held = ctx + fresh
        kept = np.maximum(held - np.array(drop), 0)
        f0, c0 = free.cpu().numpy(), int(count[0])
        count = q.kv_trim(table, up(held.astype(np.int32)), up(kept.astype(np.int32)), free, count, page_size=page)
        f1, left = step_ref.trim(tb, held, kept, f0, c0, page)
        assert int(count[0]) == left and np.array_equal(free.cpu().numpy()[:left], f1[:left])
        ctx = kept
        # every page is held by one request or free
        ids = [tb[b, :held_pages(ctx[b])] for b in range(B)] + [free.cpu().numpy()[:left]]
        assert sorted(np.concatenate(ids).tolist()) == list(range(pages))


def every(seed):
    """A call of each operator with buffers of its own -> (run, inputs to refill, outputs)."""
    rng = np.random.default_rng(seed)
    gen = torch.Generator().manual_seed(seed)
    B, T, k = 40, 300, 512
    ctx, fresh = up(rng.integers(0, 500, B).astype(np.int32)), up(rng.integers(0, 8, B).astype(np.int32))
    table = torch.full((B, 10), -1, dtype=I32, device=DEV)
    free, count = up(rng.permutation(500).astype(np.int32)), up(np.array([400], np.int32))
    plan = tuple(torch.empty(n, dtype=I32, device=DEV) for n in (B + 1, T, T, B, 1))
    free2, left = up(rng.permutation(500).astype(np.int32)), torch.empty(1, dtype=I32, device=DEV)
    count2 = up(np.array([20], np.int32))
    kept = up(np.zeros(B, np.int32))
    x, res = torch.randn(T, k, generator=gen).to(DEV), torch.randn(T, k, generator=gen).half().to(DEV)
    total = torch.empty_like(res)
    x8 = torch.empty(8, q.row_bytes(q.Q8_0, k), dtype=torch.uint8, device=DEV)
    xn = torch.empty(T, k, dtype=torch.float16, device=DEV)
    types, ns = [G.Q4_K, G.Q8_0, G.Q6_K], [100, 33, 257]
    ws = [up(G.gen_weights(t, n, k, seed + n)) for t, n in zip(types, ns)]
    ys = [torch.empty(8, n, device=DEV) for n in ns]
    a, b = (torch.randn(3, 24, k, generator=gen) / 30).half().to(DEV), torch.randn(3, 65, 24, generator=gen).half().to(DEV)
    base, y = torch.randn(T, 65, generator=gen).to(DEV), torch.zeros(T, 65, device=DEV)
    adapter = up(rng.integers(-1, 3, B).astype(np.int32))
    wsp = q.lora_workspace(x, [(a, b, y, base)], adapter)

    def run():
        q.kv_plan(table, ctx, fresh, free, count, T, out=plan)
        q.kv_trim(table, ctx, kept, free2, count2, left=left)
        q.rms_norm(x, residual=res, sum_out=total, out=xn)
        q.rms_norm(x[:8], qtype=q.Q8_0, out=x8)
        q.gemv_q8_multi(ws, types, ns, k, x8, outs=ys)
        q.lora(xn, [(a, b, y, base)], adapter, qstart=plan[0], workspace=wsp)

    pool = free2.clone()

    def refill(r):
        """New inputs; what calls read and write is as at the start, outputs are blank."""
        for o in (*plan, left, total, xn, x8, *ys, y):
            o.zero_()
        table.fill_(-1)
        free2.copy_(pool)
        g = torch.Generator().manual_seed(1000 * seed + r)
        x.copy_(torch.randn(T, k, generator=g))
        res.copy_(torch.randn(T, k, generator=g))
        base.copy_(torch.randn(T, 65, generator=g))
        ctx.copy_(torch.randint(0, 500, (B,), generator=g))
        fresh.copy_(torch.randint(0, 8, (B,), generator=g))
        adapter.copy_(torch.randint(-1, 3, (B,), generator=g))
    return run, refill, [table, *plan, free2, left, total, xn, x8, *ys, y]


def test_graph_replays_are_the_eager_results():
    run, refill, outs = every(1)
    refill(0)
    run()                                  # workspaces and code loaded
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for r in range(1, 6):
        refill(r)
        run()
        eager = [o.clone() for o in outs]
        torch.cuda.synchronize()
        refill(r)
        graph.replay()
        torch.cuda.synchronize()
        for i, (o, e) in enumerate(zip(outs, eager)):
            assert torch.equal(o, e), (r, i)


def test_on_streams_of_their_own_at_once():
    pairs = [every(s) for s in (3, 4, 5)]
    want = []
    for run, refill, outs in pairs:
        refill(7)
        run()
        want.append([o.clone() for o in outs])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in pairs]
    for _ in range(4):
        for run, refill, outs in pairs:
            refill(7)
        torch.cuda.synchronize()
        for (run, _, _), s in zip(pairs, streams):
            with torch.cuda.stream(s):
                run()
        torch.cuda.synchronize()
        for (_, _, outs), w in zip(pairs, want):
            assert all(torch.equal(o, e) for o, e in zip(outs, w))


def test_a_call_reports_its_own_launch():
    import ctypes
    paths = {line.split()[-1] for line in open("/proc/self/maps") if "libamdhip64" in line}
    hip = ctypes.CDLL(paths.pop())
    run, refill, _ = every(6)
    run()
    torch.cuda.synchronize()
    bad = hip.hipSetDevice(99)
    assert bad != 0
    run()
    assert hip.hipGetLastError() == bad
    torch.cuda.synchronize()
