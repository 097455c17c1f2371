"""GPU tests of each shape of workgroup of the attention: 64, 128 and 256 rows of the
kernel of many rows, splits longer than the page ids that a wave holds, page ids
outside the cache.  Which shape a call takes is read from its launch, so that a change
of the rule that picks it cannot quietly leave one without a test.  Bars:
test_gpu_attention_bars.py.
"""
import numpy as np
import pytest

import kv_ref as R
import test_gpu_attention as A

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import dequant_matmul_amd as q  # noqa: E402
from graph_nodes import launched  # noqa: E402
from test_gpu_attention_bars import judge, put  # noqa: E402

up, DEV = A.up, A.DEV
F32, F16 = A.DTS


def shape(c, run, rows):
    """(rows of a workgroup, splits) of the call run(), whose sequences have at most
    `rows` rows a kv head (up to 32 are always taken by the kernel of few rows)."""
    kvh = c.cache.kv_heads
    threads, (splits, y, _) = launched(run)[0]
    fits = [r for r, t in ((16, 256), (64, 256), (128, 512), (256, 512))
            if t == threads and -(-rows // r) * kvh == y and (r == 16) == (rows <= 32)]
    assert len(fits) == 1
    return fits[0], splits


def ready(c, dt):
    """The call of case c with everything on the device."""
    args = (c.cache, up(c.q).to(dt), up(c.table), up(np.array(c.ctx, np.int32)))
    kw = dict(qstart=up(c.starts), mask=up(c.mask) if c.mask is not None else None, max_q=max(c.tq),
              max_ctx=max(x + t for x, t in zip(c.ctx, c.tq)))
    return lambda: q.attention(*args, **kw)


def sample(c, b, n=10):
    """Some rows of sequence b: the first, the last and n others; three heads."""
    rng = np.random.default_rng(b)
    t = c.tq[b]
    rows = np.unique(np.concatenate([[0, t - 1], rng.integers(0, t, n)]))
    return rows, np.unique([0, c.q.shape[1] - 1, int(rng.integers(c.q.shape[1]))])


# (rows, type): kv heads, group, committed and new tokens.  The last row group holds
# waves with all, some and none of their rows.
CALLS = [(256, F16, 4, 8, (1500, 70), (251, 13)), (256, F16, 8, 8, (100,), (699,)),
         (128, F16, 8, 4, (700,), (251,)), (64, F16, 4, 4, (700,), (251,)),
         (128, F32, 8, 4, (700,), (251,)), (64, F32, 4, 4, (700,), (251,))]


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("kind", A.KINDS)
@pytest.mark.parametrize("D", [64, 80, 128])
@pytest.mark.parametrize("rows,dt,kvh,group,ctx,tq", CALLS)
def test_rows_of_a_workgroup(rows, dt, kvh, group, ctx, tq, D, kind, tree):
    c = A.Case(kind, list(ctx), list(tq), kvh, group, D, page=128, seed=rows + D, tree=tree)
    run = ready(c, dt)
    got = run()
    assert shape(c, run, max(tq) * group)[0] == rows
    for b in range(len(ctx)):
        judge(c, got, dt, b, *sample(c, b))


@pytest.mark.parametrize("dt,kvh,group,ctx,tq,rows", [(F16, 8, 4, 700, 251, 128), (F16, 4, 4, 700, 251, 64),
                                                      (F32, 4, 4, 700, 251, 64)])
@pytest.mark.parametrize("kind", A.KINDS)
def test_rows_of_a_workgroup_of_wide_heads(dt, kvh, group, ctx, tq, rows, kind):
    c = A.Case(kind, [ctx], [tq], kvh, group, 256, page=64, seed=3)
    run = ready(c, dt)
    got = run()
    assert shape(c, run, tq * group)[0] == rows
    judge(c, got, dt, 0, *sample(c, 0))


@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("D", [64, 80, 128, 256])
@pytest.mark.parametrize("rows,dt,kvh,group,ctx,tq", CALLS[:4])
def test_the_largest_values_saturate(rows, dt, kvh, group, ctx, tq, D, which):
    """Q8_0, decoded to fp16: 127 times the scale of a block whose largest value is 65504
    is 65532, past the fp16 range.  As V of a token alike for all dims and of a weight
    near 1 it comes out as 65504 (no rounding of a weight below 1 takes it higher), and
    leaves no infinity in any row; as K it does not reach other tokens' scores."""
    if D == 256 and rows == 256:
        pytest.skip("no such shape: 128 rows at most")
    c = A.Case("q8_0", list(ctx), list(tq), kvh, group, D, page=128, seed=7)
    at = ctx[0] // 2
    k, v = c.k[0].copy(), c.v[0].copy()
    (k if which == "k" else v)[at] = np.sign((k if which == "k" else v)[at]) * 65504.0
    if which == "v":
        k[at] = 0
    put(c, 0, k, v)
    if which == "k":
        c.q[c.starts[0]:c.starts[1]] *= 2.0 ** -6        # scores within a few thousand
    run = ready(c, dt)
    got = run()
    assert shape(c, run, max(tq) * group)[0] == rows
    assert torch.isfinite(got).all()
    for b in range(len(ctx)):
        judge(c, got, dt, b, *sample(c, b))


def shared(kind, B, ctx, tq, kvh, group, D, dt, columns):
    """One sequence's tokens seen by B sequences (the same pages in each row of the
    table) with new tokens' queries of their own."""
    c = A.Case(kind, [ctx], [tq], kvh, group, D, page=64, seed=B)
    assert c.cols >= columns
    rng = np.random.default_rng(B)
    rows = (rng.standard_normal((B * tq, kvh * group, D))).astype(np.float32)
    args = (c.cache, up(rows).to(dt), up(np.repeat(c.table, B, 0)), torch.full((B,), ctx, dtype=torch.int32, device=DEV))
    return c, rows, lambda: q.attention(*args, max_q=tq, max_ctx=ctx + tq)


def judge_shared(c, rows, got, dt, tq, group):
    for b in (0, len(rows) // tq // 2, len(rows) // tq - 1):
        c.q = rows[b * tq:(b + 1) * tq]
        judge(c, got[b * tq:(b + 1) * tq], dt, 0, heads=[0, c.q.shape[1] - 1])


@pytest.mark.parametrize("dt", A.DTS)
@pytest.mark.parametrize("kind", A.KINDS)
def test_more_page_ids_than_a_wave_holds(kind, dt):
    """Single tokens of 64 sequences in one split of 68 pages; the kernel fetches 64 page
    ids at a time."""
    c, rows, run = shared(kind, 64, 4300, 1, 8, 4, 64, dt, 68)
    got = run()
    assert shape(c, run, 4) == (16, 1)
    judge_shared(c, rows, got, dt, 1, 4)


@pytest.mark.parametrize("dt", A.DTS)
@pytest.mark.parametrize("kind", ["f16", "q8_0"])
def test_more_page_ids_than_a_wave_holds_many_rows(kind, dt):
    """The same with 9 new tokens each, 36 rows a kv head; three fetches."""
    c, rows, run = shared(kind, 64, 8300, 9, 8, 4, 64, dt, 130)
    got = run()
    r, splits = shape(c, run, 36)
    assert r > 16 and splits == 1
    judge_shared(c, rows, got, dt, 9, 4)


@pytest.mark.parametrize("dt", A.DTS)
@pytest.mark.parametrize("kind", A.KINDS)
@pytest.mark.parametrize("tq,ctx,kvh", [(1, 700, 2), (40, 700, 2), (40, 300, 64)])
@pytest.mark.parametrize("gone", [(0,), (1, 3), (2, 3), (-2,), (-1,), (0, 1, -2, -1)])
def test_pages_outside_the_cache(kind, dt, tq, ctx, kvh, gone):
    """Page ids outside the cache hide their tokens: the first, some, two in a row, the
    last ones (with new tokens on them), in one split and in several."""
    c = A.Case(kind, [ctx], [tq], kvh, 4, 64, seed=60 + len(gone))
    for i, col in enumerate(gone):
        col %= c.cols
        c.table[0, col] = (-1, c.pages, 2 ** 31 - 1, -2 ** 31)[i]
        c.see[0][:, 64 * col:64 * (col + 1)] = False
    run = ready(c, dt)
    got = run()
    r, splits = shape(c, run, tq * 4)
    assert (r == 16) == (tq == 1) and (splits > 1) == (ctx > 512)
    judge(c, got, dt, heads=[0, c.q.shape[1] - 1])


@pytest.mark.parametrize("dt", A.DTS)
@pytest.mark.parametrize("max_q", [2, 20])
@pytest.mark.parametrize("starts", [[0, 100, 50], [-7, 1, 2], [2, 1, 0], [5, 9, 90], [-2 ** 31, 2 ** 31 - 1, 0]])
def test_first_rows_outside_q(starts, max_q, dt):
    """Rows given to sequences out of order or outside q: what is left of them in q is
    computed, everything else keeps what it held."""
    c = A.Case("q8_0", [300, 200], [1, 1], 2, 4, 64, seed=10, tail=7)
    T, H, D = c.q.shape
    memory = torch.full((T + 6, H, D), 7.0, dtype=dt, device=DEV)
    got = memory[3:3 + T]
    q.attention(c.cache, up(c.q).to(dt), up(c.table), up(np.array(c.ctx, np.int32)),
                qstart=up(np.array(starts, np.int32)), max_q=max_q, max_ctx=301, out=got)
    free = np.ones(T, bool)
    c.starts = np.zeros(3, np.int64)
    for b in range(2):
        first = min(max(starts[b], 0), T)
        n = min(max(starts[b + 1], first), T) - first
        free[first:first + min(n, max_q)] = False
        if n:           # its first row sees the committed tokens and itself
            c.starts[b] = first
            judge(c, got, dt, b, rows=[0])
    assert (got[up(free)] == 7).all() and not (got[up(~free)] == 7).any()
    assert (memory[:3] == 7).all() and (memory[3 + T:] == 7).all()


@pytest.mark.parametrize("dt", A.DTS)
def test_the_most_sequences(dt):
    """65535 sequences of one token, all over the same two pages."""
    B, kvh, group, D = 65535, 1, 2, 64
    c = A.Case("q8_0", [69], [1], kvh, group, D, seed=80)
    rows = np.random.default_rng(81).standard_normal((B, kvh * group, D)).astype(np.float32)
    got = q.attention(c.cache, up(rows).to(dt), up(c.table).expand(B, -1).contiguous(),
                      torch.full((B,), 69, dtype=torch.int32, device=DEV), max_ctx=70)
    for b in (0, 1, 32767, 32768, 65534):
        c.q = rows[b:b + 1]
        judge(c, got[b:b + 1], dt)


@pytest.mark.parametrize("dt", A.DTS)
def test_the_most_row_groups(dt):
    """1024 kv heads with so many rows each that the groups of them fill a dimension of
    the launch; twice as many are refused."""
    kvh, D = 1024, 8
    tq = 4032
    c = A.Case("f16", [0], [tq], kvh, 1, D, seed=82)
    run = ready(c, dt)
    got = run()
    assert launched(run)[0][1][1] > 65535 // 2 or dt == F16
    rows = np.array([0, 1, 63, 64, 2000, 4031])
    judge(c, got, dt, rows=rows, heads=[0, 511, 1023])
    x = torch.zeros(17 * tq, kvh, D, dtype=dt, device=DEV)
    with pytest.raises((ValueError, q.QmmError)):
        q.attention(c.cache, x, up(c.table), up(np.array([0], np.int32)), max_ctx=64 * c.cols)
