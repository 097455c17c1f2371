"""The cache operators together, as a decoder uses them: a layer between its
projections, prompt chunks and single tokens against one causal pass, drafted
trees verified and committed, captured graphs replayed, other streams, caches
past 4 GiB.
"""
import numpy as np
import pytest

import kv_ref as R
import oracle
import qmm_inputs as G
import test_gpu_attention as A

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import dequant_matmul_amd as q  # noqa: E402

DEV = "cuda:0"
up = A.up


def i32(*v):
    return up(np.array(v, np.int32))


def test_layer_between_its_projections():
    """One token through q | k | v (a stage of the decode pass), rotation, cache,
    attention and o, with 4-bit K-quant weights, on top of 100 cached tokens.
    Bar: the GEMVs' 2e-5 of sum |w x| passes through rotation and attention; q, k
    off by 2e-5 move a score by 4e-5 sum |q k| scale and its weight by that
    factor, and K and V may round to the neighbouring code (half a step of the
    block each, one code in a hundred of a single token): so the attention is
    checked on the values that the cache really holds, within its own bar, and the
    projections and the cached row apart."""
    rng = np.random.default_rng(5)
    hid, H, K, D, L = 1024, 8, 2, 128, 100
    wq, wk, wv, wo = (G.gen_weights(G.Q4_K, n, hid, 40 + i) for i, n in enumerate((H * D, K * D, K * D, hid)))
    x = G.gen_x(hid, 1, 50)[0]
    y = torch.empty((H + 2 * K) * D, device=DEV)
    yq, yk, yv = y[:H * D], y[H * D:(H + K) * D], y[(H + K) * D:]
    xd, att, out = up(x), torch.empty(1, H, D, device=DEV), torch.empty(hid, device=DEV)
    dq, dk, dv, do = map(up, (wq, wk, wv, wo))
    q.gemv_pass([(dq, G.Q4_K, H * D, hid, xd, yq, 0), (dk, G.Q4_K, K * D, hid, xd, yk, 0), (dv, G.Q4_K, K * D, hid, xd, yv, 0)])
    freqs, m = q.rope_freqs(D, 500000.0)
    cache = q.KVCache(q.Q8_0, K, D, 3)
    table = i32(2, 0).reshape(1, 2)
    kp, vp = rng.standard_normal((2, L, K, D)).astype(np.float32)
    pos = np.arange(L)
    slots = np.array([2, 0])[pos // 64] * 64 + pos % 64
    q.kv_append(cache, up(kp), up(vp), up(slots.astype(np.int32)))
    cs = q.rope_angles(i32(L), freqs.to(DEV), m)
    q3 = yq.view(1, H, D)
    q.rope(q3, cs, out=q3)
    q.kv_append(cache, yk.view(1, K, D), yv.view(1, K, D), i32(0 * 64 + L - 64), cs=cs)
    q.attention(cache, q3, table, i32(L), out=att)
    q.gemv(do, G.Q4_K, hid, hid, att.view(1, -1), out=out.view(1, -1))
    # the projections and the rotation
    c64 = R.angles([L], freqs.numpy(), m)
    ref, a = oracle.gemv(G.Q4_K, wq, H * D, hid, x[None])
    want = R.rotate(ref.reshape(1, H, D).astype(np.float64), c64, False)
    size = np.abs(a.reshape(1, H, D))
    size = size + np.roll(size, D // 2, -1)
    assert np.all(np.abs(q3.cpu().numpy() - want) <= 3e-5 * size)
    # the attention over what the cache holds, and the o projection of it
    held = q.kv_read(cache, up(np.append(slots, L - 64).astype(np.int32)))
    k, v = (t.cpu().numpy().astype(np.float64) for t in held)
    c = A.Case.__new__(A.Case)
    c.ctx, c.tq, c.D, c.starts, c.q = [L], [1], D, np.array([0, 1]), q3.cpu().numpy()
    c.k, c.v, c.see = [k], [v], [np.ones((1, L + 1), bool)]
    c.check(att, torch.float32)
    ref, a = oracle.gemv(G.Q4_K, wo, hid, hid, att.cpu().numpy().reshape(1, -1))
    assert np.all(np.abs(out.cpu().numpy() - ref) <= 2e-5 * a)
    # the new token's own K and V rows: the projections within a code step
    refk, ak = oracle.gemv(G.Q4_K, wk, K * D, hid, x[None])
    rk = R.rotate(refk.reshape(1, K, D).astype(np.float64), c64, False)
    step = np.abs(rk).reshape(K, D // 32, 32).max(-1) / 127
    assert np.all(np.abs(k[-1].reshape(K, D // 32, 32) - rk.reshape(K, D // 32, 32)) <= 0.51 * step[..., None] + 2.0 ** -11 * np.abs(rk).max()
                  + 4e-5 * ak.max())


@pytest.mark.parametrize("kind", A.KINDS)
@pytest.mark.parametrize("dt", A.DTS)
def test_chunks_and_single_tokens_make_one_causal_pass(kind, dt):
    """A prompt in chunks of 100, 64 and 37 and then single tokens: each output is
    that of one causal attention over all tokens, whatever the cut."""
    rng = np.random.default_rng(3)
    K, g, D, n = 2, 4, 128, 206
    k, v = rng.standard_normal((2, n, K, D)).astype(np.float32)
    x = rng.standard_normal((n, K * g, D)).astype(np.float32)
    cache = q.KVCache(R.TYPES[kind], K, D, 4)
    cache.k.fill_(255)
    cache.v.fill_(255)
    table = i32(3, 1, 0, 2).reshape(1, 4)
    slots = up((table.cpu().numpy()[0][np.arange(n) // 64] * 64 + np.arange(n) % 64).astype(np.int32))
    kd, vd, xd = up(k), up(v), up(x).to(dt)
    outs, at = [], 0
    for step in (100, 64, 37, 1, 1, 1, 1, 1):
        s = slice(at, at + step)
        q.kv_append(cache, kd[s], vd[s], slots[s])
        outs.append(q.attention(cache, xd[s], table, i32(at)))
        at += step
    c = A.Case.__new__(A.Case)
    c.ctx, c.tq, c.D, c.starts, c.q = [0], [n], D, np.array([0, n]), x
    c.k, c.v, c.see = [R.stored(k, kind)], [R.stored(v, kind)], [np.tril(np.ones((n, n), bool))]
    c.check(torch.cat(outs), dt)


@pytest.mark.parametrize("kind", A.KINDS)
def test_drafted_tree_is_verified_and_committed(kind):
    """The rows of a path through the tree give what the same tokens give one
    after the other; once moved down, the next token sees them as if the rest had
    never been drafted."""
    rng = np.random.default_rng(8)
    K, g, D, ctx, n = 2, 4, 64, 75, 40
    par, see = R.tree(rng, n)
    path = [max(range(n), key=lambda i: see[i].sum())]
    while par[path[0]] >= 0:
        path.insert(0, par[path[0]])
    depth = see.sum(1) - 1
    k, v = rng.standard_normal((2, ctx + n, K, D)).astype(np.float32)
    x = rng.standard_normal((n, K * g, D)).astype(np.float32)
    freqs, m = q.rope_freqs(D)
    pages = [4, 0, 3]

    def slot(p):
        p = np.asarray(p)
        return up((np.array(pages)[p // 64] * 64 + p % 64).astype(np.int32))

    def fresh():
        c = q.KVCache(R.TYPES[kind], K, D, 5)
        c.k.fill_(255)
        c.v.fill_(255)
        cs = q.rope_angles(up(np.arange(ctx, dtype=np.int32)), freqs.to(DEV), m)
        q.kv_append(c, up(k[:ctx]), up(v[:ctx]), slot(np.arange(ctx)), cs=cs)
        return c
    table = i32(*pages).reshape(1, 3)
    # the tree at once
    c = fresh()
    cs = q.rope_angles(up((ctx + depth).astype(np.int32)), freqs.to(DEV), m)
    q.kv_append(c, up(k[ctx:]), up(v[ctx:]), slot(ctx + np.arange(n)), cs=cs)
    qt = q.rope(up(x), cs)
    got = q.attention(c, qt, table, i32(ctx), mask=up(R.words(see)))[path]
    # its path, token by token
    one = fresh()
    for d, node in enumerate(path):
        cs1 = q.rope_angles(i32(ctx + d), freqs.to(DEV), m)
        q.kv_append(one, up(k[ctx + node][None]), up(v[ctx + node][None]), slot([ctx + d]), cs=cs1)
        ref = q.attention(one, q.rope(up(x[node][None]), cs1), table, i32(ctx + d))
        # the same scores and values in another order of summing: 2^-18 of sums of
        # |p v| <= max |v| and of scores, as in the attention's own bar, twice
        assert (got[d] - ref[0]).abs().max() <= 2 * 2.0 ** -16 * np.abs(v).max()
    # committed
    q.kv_move(c, slot(ctx + np.array(path))[None].contiguous(), slot(ctx + np.arange(len(path)))[None].contiguous())
    upto = slot(np.arange(ctx + len(path)))
    for a, b in zip(q.kv_read(c, upto), q.kv_read(one, upto)):
        assert torch.equal(a, b)
    nxt = up(x[:1])
    p = i32(ctx + len(path) - 1)
    assert torch.equal(q.attention(c, nxt, table, p), q.attention(one, nxt, table, p))


@pytest.mark.parametrize("dt", A.DTS)
def test_graph_replays_match_eager(dt):
    """Every entry point in one captured graph (decode in splits and whole, a
    tree, a chunk), replayed with new inputs, lengths and pages between eager work
    and synchronizations."""
    rng = np.random.default_rng(21)
    K, g, D, cap, B = 2, 4, 128, 4096, 2
    freqs = q.rope_freqs(D)[0].to(DEV)
    cols = cap // 64
    pages = B * cols + 1
    cache, eager = (q.KVCache(q.Q8_0, K, D, pages) for _ in range(2))
    fill = up(rng.standard_normal((pages * 64, K, D)).astype(np.float16))
    every = torch.arange(pages * 64, dtype=torch.int32, device=DEV)
    for c in (cache, eager):
        q.kv_append(c, fill, fill.flip(0), every)
    T = 40
    pos, slots = (torch.empty(T, dtype=torch.int32, device=DEV) for _ in range(2))
    kv = torch.empty(2, T, K, D, dtype=dt, device=DEV)
    x = torch.empty(T, K * g, D, dtype=dt, device=DEV)
    table = torch.empty(B, cols, dtype=torch.int32, device=DEV)
    ctx = torch.empty(B, dtype=torch.int32, device=DEV)
    starts = torch.empty(B + 1, dtype=torch.int32, device=DEV)
    mask = torch.empty(T, 1, dtype=torch.int64, device=DEV)
    src, dst = (torch.empty(2, 5, dtype=torch.int32, device=DEV) for _ in range(2))

    def load(r):
        rr = np.random.default_rng(100 + r)
        kv.copy_(up(rr.standard_normal((2, T, K, D)).astype(np.float32)))
        x.copy_(up(rr.standard_normal((T, K * g, D)).astype(np.float32)))
        pos.copy_(up(rr.integers(0, 5000, T).astype(np.int32)))
        perm = rr.permutation(pages * 64).astype(np.int32)
        slots.copy_(up(perm[:T]))
        src.copy_(up(perm[T:T + 10].reshape(2, 5)))
        dst.copy_(up(perm[T + 10:T + 20].reshape(2, 5)))
        table.copy_(up(rr.permutation(pages)[:B * cols].reshape(B, cols).astype(np.int32)))
        ctx.copy_(up(rr.integers(0, 3900, B).astype(np.int32)))
        a = int(rr.integers(1, 30))
        starts.copy_(up(np.array([0, a, a + int(rr.integers(1, 30 - a + 10))], np.int32).clip(0, T)))
        mask.copy_(up(rr.integers(-2 ** 62, 2 ** 62, (T, 1))))

    def run(c, ws):
        cs = q.rope_angles(pos, freqs)
        xr = q.rope(x, cs)
        q.kv_append(c, kv[0], kv[1], slots, cs=cs)
        outs = [cs, xr]
        for i, kw in enumerate((dict(mask=mask, max_q=T), dict(max_q=T), dict(max_q=1), dict(max_q=T, max_ctx=448))):
            o = torch.zeros_like(x)
            outs.append(q.attention(c, xr, table, ctx, qstart=starts, out=o, workspace=ws[i], **kw))
        q.kv_move(c, src, dst)
        outs += list(q.kv_read(c, every, torch.float16))
        return outs
    ws = [q.attention_workspace(cache, x, table, max_q=mq, max_ctx=mc) for mq, mc in ((T, None), (T, None), (1, None), (T, 448))]
    assert ws[0].numel() > 0
    load(0)
    run(cache, ws)
    run(eager, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(cache, ws)
    other = [torch.empty_like(w) for w in ws]
    for c in (cache, eager):            # the same bytes on both sides
        q.kv_append(c, fill, fill.flip(0), every)
    for r in range(1, 5):
        load(r)
        graph.replay()
        want = run(eager, other)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), "replay %d" % r


def test_two_streams_at_once():
    """Two calls in flight on streams of their own, each with its own workspace,
    while the default stream is busy."""
    c = A.Case("q8_0", [5000, 3000], [1, 1], 2, 4, 128, seed=31)
    args = (c.cache, up(c.q), up(c.table), i32(*c.ctx))
    want = q.attention(*args, max_q=1)
    torch.cuda.synchronize()
    busy = torch.randn(4096, 4096, device=DEV)
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for rep in range(4):
        busy = busy @ busy * 1e-3
        for s in streams:
            with torch.cuda.stream(s):
                got.append(q.attention(*args, max_q=1))
    torch.cuda.synchronize()
    for o in got:
        assert torch.equal(o, want)
    c.check(want, torch.float32)


@pytest.mark.parametrize("dt", A.DTS)
@pytest.mark.parametrize("tree", [False, True])
def test_many_rows_over_a_long_context(dt, tree):
    """Row groups of every size with the tokens split, ragged."""
    c = A.Case("q8_0", [4000, 1, 2500], [60, 33, 12], 1, 4, 128, seed=32, tree=tree)
    c.check(c.run(dt), dt)
    c = A.Case("f16", [2100], [150], 1, 8, 64, seed=33, tree=tree, page=256)
    c.check(c.run(dt), dt)


def test_cache_past_4_gib():
    """Byte offsets past 32 bits: rows at the end of a 5 GiB buffer."""
    K, D, page = 8, 128, 256
    pages = 5 * (1 << 30) // q.lib.qkv_page_bytes(q.F16, K, D, page)
    cache = q.KVCache(q.F16, K, D, pages, page_size=page)
    rng = np.random.default_rng(9)
    n = 300
    k, v = rng.standard_normal((2, n, K, D)).astype(np.float16)
    table = np.array([pages - 1, 0], np.int32)
    slots = up((table[np.arange(n) // page] * page + np.arange(n) % page).astype(np.int32))
    q.kv_append(cache, up(k), up(v), slots)
    for got, want in zip(q.kv_read(cache, slots, torch.float16), (k, v)):
        assert np.array_equal(got.cpu().numpy(), want)
    x = rng.standard_normal((1, 32, D)).astype(np.float32)
    out = q.attention(cache, up(x), up(table.reshape(1, 2)), i32(n - 1))
    ref = R.attend(x.astype(np.float64), k.astype(np.float64), v.astype(np.float64), np.ones((1, n), bool), D ** -0.5)
    assert np.abs(out.cpu().numpy() - ref).max() <= 2.0 ** -16 * np.abs(v).max()
    q.kv_move(cache, slots[:3][None].contiguous(), slots[297:][None].contiguous())
    assert np.array_equal(q.kv_read(cache, slots[297:], torch.float16)[0].cpu().numpy(), k[:3])
