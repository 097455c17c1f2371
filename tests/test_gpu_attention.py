"""GPU tests of attention over the paged KV cache against a 64-bit reference on
the values that the cache holds.

Bars, relative to A = sum_j p_j |v_j| of the reference (the size of what is
summed; the output itself cancels) plus the score error's effect.  A score s =
scale q.k, in units of the exponent, has the error e_s = c 2^-k sum_d |scale q_d
k_d|, and moves a weight by that factor: at most 2 e_s A.
  float32: q and the weights in two fp16 parts, 2^-21 each; fp32 sums of up to
    256 products a block of the matrix cores and 64 tokens a tile: c 2^-k = 2^-19
    for the scores (parts, sums and scales), and 2^-18 of A for the weights,
    their sums (a tree over tiles and splits) and the exponential (2^-22).
  float16, few rows: q exact; weights rounded once to fp16 (2^-11), the output
    rounded once (2^-11 of it): 2^-19 for the scores, 2^-10 of A.
  float16 chunks: K and V rounded to fp16 as well: 2^-11 for the scores, 3 2^-11
    of A with the weights' rounding and 2^-11 for the output.
Weights below 2^-14 of the fp16 range lose relative accuracy: 2^-24 of the
largest |v| per token in all (fp16), 2^-30 (float32, two parts).
"""
import numpy as np
import pytest

import kv_ref as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import dequant_matmul_amd as q  # noqa: E402

DEV = "cuda:0"
KINDS = ["f16", "q8_0", "q4_0"]


def up(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


class Case:
    """Sequences of ctx committed and tq new tokens in a shuffled paged cache
    whose unused bytes are all ones."""

    def __init__(self, kind, ctx, tq, kvh, group, D, page=64, seed=0, spread=1.0, tree=False, tail=0, vscale=1.0):
        rng = np.random.default_rng(seed)
        self.rng, self.kind, self.ctx, self.tq, self.D, self.page = rng, kind, ctx, tq, D, page
        B = len(ctx)
        self.cols = max(1, max(-(-(c + t) // page) for c, t in zip(ctx, tq)))
        self.pages = B * self.cols + 2
        self.cache = q.KVCache(R.TYPES[kind], kvh, D, self.pages, page_size=page)
        self.cache.k.fill_(255)
        self.cache.v.fill_(255)
        self.table = rng.permutation(self.pages)[:B * self.cols].reshape(B, self.cols).astype(np.int32)
        self.k, self.v, self.see = [], [], []
        for b in range(B):
            n = ctx[b] + tq[b]
            p = np.arange(n)
            slots = self.table[b, p // page] * page + p % page
            k, v = rng.standard_normal((2, n, kvh, D)).astype(np.float32)
            v *= vscale
            if n:
                q.kv_append(self.cache, up(k), up(v), up(slots.astype(np.int32)))
            self.k.append(R.stored(k, kind))
            self.v.append(R.stored(v, kind))
            new = R.tree(rng, tq[b])[1] if tree and tq[b] else np.tril(np.ones((tq[b], tq[b]), bool))
            self.see.append(np.concatenate([np.ones((tq[b], ctx[b]), bool), new], 1))
        self.starts = np.concatenate([[0], np.cumsum(tq)]).astype(np.int32)
        self.T = int(self.starts[-1]) + tail
        self.q = (spread * rng.standard_normal((self.T, kvh * group, D))).astype(np.float32)
        self.mask = None
        if tree:
            w = max(1, -(-max(tq) // 64))
            self.mask = np.zeros((self.T, w), np.int64)
            for b in range(B):
                self.mask[self.starts[b]:self.starts[b + 1]] = R.words(self.see[b][:, ctx[b]:], w)

    def run(self, dt, **kw):
        args = dict(qstart=up(self.starts), mask=up(self.mask) if self.mask is not None else None,
                    max_q=max(self.tq), max_ctx=max(c + t for c, t in zip(self.ctx, self.tq)))
        args.update(kw)
        qd = up(self.q).to(dt)
        return q.attention(self.cache, qd, up(self.table), up(np.array(self.ctx, np.int32)), **args)

    def check(self, got, dt, scale=None):
        scale = self.D ** -0.5 if scale is None else scale
        qd = up(self.q).to(dt).cpu().numpy().astype(np.float64)
        got = got.cpu().numpy().astype(np.float64)
        for b in range(len(self.ctx)):
            rows = slice(self.starts[b], self.starts[b + 1])
            if self.tq[b] == 0:
                continue
            x, k, v, see = qd[rows], self.k[b], self.v[b], self.see[b]
            ref = R.attend(x, k, v, see, scale)
            size = R.attend(x, k, np.abs(v), see, scale)
            g = x.shape[1] // k.shape[1]
            es = np.stack([(np.abs(scale * x[:, h]) @ np.abs(k[:, h // g]).T * see).max(-1) for h in range(x.shape[1])], 1)
            most = np.abs(v).max(initial=0)
            if dt == torch.float32:
                tol = (2.0 ** -18 + 2 * 2.0 ** -19 * es[..., None]) * size + 2.0 ** -30 * most * len(k)
            else:
                tol = (2.0 ** -9 + 2 * 2.0 ** -11 * es[..., None]) * size + 2.0 ** -24 * most * len(k)
            bad = ~(np.abs(got[rows] - ref) <= tol)
            assert not bad.any(), "sequence %d: %d of %d off, worst %.3g of the bar" % (
                b, bad.sum(), bad.size, np.nanmax(np.abs(got[rows] - ref) / tol))
        return got


DTS = [torch.float32, torch.float16]


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [8, 64, 80, 96, 128, 200, 256])
def test_single_tokens(kind, D, dt):
    """Lengths around tiles, pages and the end of the committed tokens; one
    token over an empty context attends to itself alone."""
    c = Case(kind, [0, 1, 62, 63, 64, 127, 128, 300], [1] * 8, 2, 4, D, page=128, seed=D)
    c.check(c.run(dt), dt)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("group", [1, 2, 7, 8, 16, 40])
def test_heads_per_kv_head(kind, group, dt):
    c = Case(kind, [131, 5], [1, 3], 3, group, 64, seed=group)
    c.check(c.run(dt), dt)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("tq", [2, 13, 61, 64, 65, 130])
def test_trees(kind, tq, dt):
    c = Case(kind, [0, 37, 500, 64], [tq, max(1, tq - 5), 1, tq], 2, 4, 128 if tq < 64 else 64, seed=tq, tree=True)
    c.check(c.run(dt), dt)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [64, 80, 128, 256])
def test_chunks(kind, D, dt):
    """Prompt chunks from an empty cache and on top of one, odd lengths."""
    c = Case(kind, [0, 203, 64, 0], [129, 200, 64, 1], 2, 4, D, page=64, seed=D)
    c.check(c.run(dt), dt)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("kind", KINDS)
def test_long_context_in_many_splits(kind, dt):
    c = Case(kind, [9001, 40], [1, 1], 2, 4, 128, page=256, seed=1)
    ws = q.attention_workspace(c.cache, up(c.q).to(dt), up(c.table), max_q=1, max_ctx=9002)
    assert ws.numel() > 0
    ws.fill_(255)                                   # what a workspace holds before does not matter
    a = c.run(dt, workspace=ws)
    c.check(a, dt)
    ws.fill_(0)
    assert torch.equal(a, c.run(dt, workspace=ws))  # the same bits again


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("spread", [1e-6, 30.0, 3000.0])
def test_sharp_and_flat_softmax(spread, dt):
    """Scores from all alike to one token taking all."""
    c = Case("q8_0", [700], [5], 2, 4, 128, seed=3, spread=spread, vscale=20.0)
    c.check(c.run(dt), dt)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("vscale", [1e-4, 1000.0])
@pytest.mark.parametrize("kind", KINDS)
def test_value_ranges(kind, vscale, dt):
    c = Case(kind, [150], [3], 1, 4, 64, seed=4, vscale=vscale)
    got = c.run(dt)
    if vscale > 1 or dt == torch.float32:
        c.check(got, dt)
    else:
        # outputs near 1e-5 are fp16 subnormals: steps of 2^-24
        ref = R.attend(up(c.q).to(dt).cpu().numpy().astype(np.float64), c.k[0], c.v[0], c.see[0], 64 ** -0.5)
        assert np.all(np.abs(got.cpu().numpy() - ref) <= 2.0 ** -9 * np.abs(c.v[0]).max() + 2.0 ** -25)


@pytest.mark.parametrize("scale", [0.0, -0.3, 1.7])
@pytest.mark.parametrize("dt", DTS)
def test_scale(scale, dt):
    c = Case("q8_0", [100], [4], 1, 4, 64, seed=5)
    c.check(c.run(dt, scale=scale), dt, scale)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("kind", KINDS)
def test_rows_that_see_nothing(kind, dt):
    c = Case(kind, [0, 0], [5, 70], 2, 4, 64, seed=6, tree=True)
    for b, r in ((0, 2), (0, 4), (1, 69)):
        c.mask[c.starts[b] + r] = 0
        c.see[b][r] = False
    got = c.check(c.run(dt), dt)
    assert not got[2].any() and not got[4].any() and not got[74].any()


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("kind", KINDS)
def test_tokens_past_the_mask_words_are_not_seen(kind, dt):
    c = Case(kind, [33], [100], 1, 4, 64, seed=7, tree=True)
    c.mask = c.mask[:, :1].copy()
    c.see[0][:, 33 + 64:] = False
    c.check(c.run(dt), dt)


@pytest.mark.parametrize("dt", DTS)
def test_rows_of_no_sequence_are_left(dt):
    """A padded batch: an empty sequence, rows behind the last one, new tokens past max_q."""
    c = Case("q8_0", [30, 50, 20], [2, 0, 9], 2, 4, 64, seed=8, tail=5)
    out = torch.full(c.q.shape, 7.0, dtype=dt, device=DEV)
    c.check(c.run(dt, out=out), dt)
    assert (out[11:] == 7).all()
    out.fill_(7)
    c.run(dt, out=out, max_q=4)
    assert (out[6:] == 7).all() and not (out[:6] == 7).all()
    # the same in several splits
    c = Case("q8_0", [3000, 50, 2000], [2, 0, 3], 2, 4, 64, seed=9, tail=5)
    out.resize_(c.q.shape).fill_(7)
    c.check(c.run(dt, out=out), dt)
    assert (out[5:] == 7).all()


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("pad", [6, 40])
@pytest.mark.parametrize("bits", [0xffff, 0x7d55, 0x7c00, 0x7bff])
def test_padded_tokens_never_appended(kind, dt, tree, pad, bits):
    """Equal shares of which the last rows are padding whose K and V were never
    written: NaN (quiet or signalling), infinity or the largest number lie there, and the rows before
    them (which do not see them) are what they are without."""
    c = Case(kind, [5, 64, 100], [4, 1, 5], 2, 4, 128, page=256, seed=pad, tree=tree, vscale=2.0 ** -6)
    clean = q.KVCache(R.TYPES[kind], 2, 128, c.pages, page_size=256)
    fill = up(np.full(c.cache.k.numel() // 2, bits, np.uint16).view(np.int16)).view(torch.uint8)
    clean.k.copy_(fill.view_as(clean.k))
    clean.v.copy_(fill.view_as(clean.v))
    for b, (ctx, t) in enumerate(zip(c.ctx, c.tq)):
        p = np.arange(ctx + t)
        slots = up((c.table[b, p // 256] * 256 + p % 256).astype(np.int32))
        rows = q.kv_read(c.cache, slots)
        q.kv_append(clean, *rows, slots)
        # the values of a quantized cache need not be its fixed points
        c.k[b], c.v[b] = (x.cpu().numpy().astype(np.float64) for x in q.kv_read(clean, slots))
    c.cache = clean
    at = np.concatenate([b * pad + np.arange(t) for b, t in enumerate(c.tq)])
    rows = np.zeros((3 * pad,) + c.q.shape[1:], np.float32)
    rows[at] = c.q
    mask = None
    if tree:
        words = np.zeros((3 * pad, 1), np.int64)
        words[at] = c.mask
        mask = up(words)
    got = q.attention(clean, up(rows).to(dt), up(c.table), up(np.array(c.ctx, np.int32)), mask=mask)
    c.check(got[up(at)], dt)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("tq", [1, 50])
@pytest.mark.parametrize("which", ["k", "v"])
def test_the_largest_stored_values(kind, dt, tq, which):
    """A stored 65504 (an infinity, clamped) in one token: it stays finite, also
    decoded (127 times the fp16 scale of a Q8_0 block is 65532), and rows that do
    not see its token do not feel it."""
    c = Case(kind, [70, 40], [tq, tq], 2, 4, 64, seed=20)
    slots, k, v = [], [], []
    for b in range(2):
        p = 30 + 45 * (tq > 1) + b            # the second sequence's is a new token if there are many
        k1, v1 = R.stored(c.k[b][p:p + 1], kind).copy(), R.stored(c.v[b][p:p + 1], kind).copy()
        (k1 if which == "k" else v1)[0, :, 3] = np.inf
        (k1 if which == "k" else v1)[0, 1, 40] = -np.inf
        k.append(k1)
        v.append(v1)
        slots.append(int(c.table[b, p // 64] * 64 + p % 64))
        at = torch.tensor([slots[-1]], dtype=torch.int32, device=DEV)
        q.kv_append(c.cache, up(k1.astype(np.float32)), up(v1.astype(np.float32)), at)
        for mine, got in zip((c.k, c.v), q.kv_read(c.cache, at)):
            mine[b][p] = got[0].cpu().numpy()
            assert np.isfinite(mine[b][p]).all() and (which == "kv"[mine is c.v]) == (np.abs(mine[b][p]).max() > 65000)
    c.check(c.run(dt), dt)


@pytest.mark.parametrize("dt", DTS)
def test_bad_indices_stay_inside(dt):
    """Page ids outside the cache hide their tokens; lengths past the table end
    there; negative ones are empty."""
    c = Case("q8_0", [300, 200], [1, 1], 2, 4, 64, seed=10)
    whole = c.table.copy()
    c.table[0, 1], c.table[0, 3] = -1, c.pages
    c.see[0][:, 64:128] = False
    c.see[0][:, 192:256] = False
    c.check(c.run(dt), dt)
    c.table = whole
    ctx = up(np.array([1 << 30, -5], np.int32))
    got = q.attention(c.cache, up(c.q).to(dt), up(c.table), ctx, qstart=up(c.starts), max_q=1, max_ctx=301)
    assert torch.isfinite(got[1]).all()
    for starts in ([0, 100, 50], [-7, 1, 2], [2, 1, 0], [5, 9, 90]):
        got = q.attention(c.cache, up(c.q).to(dt), up(c.table), up(np.array(c.ctx, np.int32)),
                          qstart=up(np.array(starts, np.int32)), max_q=2, max_ctx=301)
    torch.cuda.synchronize()


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("kind", KINDS)
def test_non_finite_queries_stay_in_their_row(kind, dt):
    c = Case(kind, [100], [6], 1, 4, 64, seed=11)
    clean = c.run(dt)
    c.q[2, 1, 5], c.q[4, 3, 0] = np.nan, np.inf
    got = c.run(dt)
    hit = torch.zeros(got.shape[:2], dtype=torch.bool, device=DEV)
    hit[2, 1] = hit[4, 3] = True
    assert torch.equal(got[~hit], clean[~hit])


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("tq", [2, 40])
def test_a_query_that_is_not_a_number_stays_one(kind, dt, tq):
    """Also where a sequence is taken in several splits; its neighbours are as without it."""
    c = Case(kind, [3000], [tq], 1, 4, 64, seed=12)
    clean = c.run(dt)
    c.q[1, 2, 5] = np.nan
    got = c.run(dt)
    assert torch.isnan(got[1, 2]).all()
    hit = torch.zeros(got.shape[:2], dtype=torch.bool, device=DEV)
    hit[1, 2] = True
    assert torch.equal(got[~hit], clean[~hit])


@pytest.mark.parametrize("dt", DTS)
def test_strided_rows_and_uniform_sequences(dt):
    c = Case("q4_0", [90, 91, 92], [2, 2, 2], 2, 4, 128, seed=12)
    H, D = c.q.shape[1:]
    wide = torch.zeros(c.T, 2 * H * D, dtype=dt, device=DEV)
    view = wide[:, H * D:].unflatten(1, (H, D))
    view.copy_(up(c.q))
    outw = torch.full((c.T, H * D + 64), 7.0, dtype=dt, device=DEV)
    out = outw[:, 64:].unflatten(1, (H, D))
    ctx = up(np.array(c.ctx, np.int32))
    q.attention(c.cache, view, up(c.table), ctx, out=out)
    c.check(out, dt)
    assert (outw[:, :64] == 7).all()
    # given starts and the same bound on the new tokens it is the same call;
    # without the bound other kernels may run, within the same bar
    assert torch.equal(out, q.attention(c.cache, up(c.q).to(dt), up(c.table), ctx, qstart=up(c.starts), max_q=2))
    c.check(q.attention(c.cache, up(c.q).to(dt), up(c.table), ctx, qstart=up(c.starts)), dt)


def test_nothing_to_do():
    c = Case("q8_0", [10], [1], 1, 1, 64)
    e = torch.empty(0, 1, 64, device=DEV)
    none = torch.zeros(0, dtype=torch.int32, device=DEV)
    assert q.attention(c.cache, e, none.reshape(0, 1), none).shape == (0, 1, 64)
    # no columns: nothing is seen
    z = q.attention(c.cache, torch.ones(1, 1, 64, device=DEV), torch.zeros(1, 0, dtype=torch.int32, device=DEV),
                    up(np.array([10], np.int32)))
    assert not z.any()


def test_refusals():
    c = Case("q8_0", [900], [1], 2, 4, 64)
    x, tab, ctx = up(c.q), up(c.table), up(np.array([900], np.int32))
    out = torch.full_like(x, 7.0)
    small = torch.empty(16, dtype=torch.uint8, device=DEV)
    for kw in (dict(mask=torch.ones(1, 1, dtype=torch.int32, device=DEV)), dict(mask=torch.ones(2, 1, dtype=torch.int64, device=DEV)),
               dict(mask=torch.ones(1, 0, dtype=torch.int64, device=DEV)), dict(qstart=ctx), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(max_q=-1), dict(max_ctx=-1), dict(workspace=small),
               dict(workspace=small.float())):
        with pytest.raises((ValueError, q.QmmError)):
            q.attention(c.cache, x, tab, ctx, out=out, **kw)
    for args in ((x.double(), tab, ctx), (x[:, :3], tab, ctx), (x, tab.long(), ctx), (x, tab, ctx.long()),
                 (x[..., :32], tab, ctx), (x.transpose(0, 1), tab, ctx), (x, tab[0], ctx), (x, tab, ctx[:0])):
        with pytest.raises((ValueError, q.QmmError)):
            q.attention(c.cache, *args, out=out if args[0] is x else None)
    with pytest.raises(ValueError):
        q.attention(c.cache, x, tab, ctx, out=out.half())
    assert (out == 7).all()
