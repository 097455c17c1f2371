"""Block tables, slots and positions (kv_plan) and pages given back (kv_trim)
against the definition, whole numbers equal; what lies around the outputs stays."""
import numpy as np
import pytest

import step_ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import dequant_matmul_amd as q  # noqa: E402

DEV = "cuda:0"
MOST = 2 ** 31 - 1


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def guarded(n):
    """(a tensor of n entries, the buffer around it)."""
    buf = torch.full((n + 32,), 77, dtype=torch.int32, device=DEV)
    return buf[16:16 + n], buf


def intact(buf):
    b = buf.cpu()
    return bool((b[:16] == 77).all()) and bool((b[-16:] == 77).all())


def check_plan(table, ctx, fresh, free, count, tokens, page, inplace=False):
    want = step_ref.plan(table, ctx, fresh, free, count, tokens, page)
    B = len(ctx)
    made = [guarded(n) for n in (B + 1, tokens, tokens, B, 1)]
    t = torch.full((table.size + 32,), 77, dtype=torch.int32, device=DEV)
    tab = t[16:16 + table.size].view(table.shape)
    tab.copy_(dev(table))
    c, f = dev([count]), dev(free)
    out = [m[0] for m in made]
    if inplace:
        out[4] = c
    got = q.kv_plan(tab, dev(ctx), None if fresh is None else dev(fresh), f, c, tokens, page_size=page, out=tuple(out))
    torch.cuda.synchronize()
    assert intact(t) and all(intact(m[1]) for m in made)
    for name, g, w in zip(("table", "qstart", "slots", "pos", "granted"), (tab, *got), want):
        assert np.array_equal(g.cpu().numpy(), w), name
    assert int(got[4][0]) == want[5]
    assert np.array_equal(f.cpu().numpy(), free) and (inplace or int(c[0]) == count)
    return tab, got


def problem(rng, B, ctx, tq, page, spare=None, waits=0.2, cols=None):
    have = rng.integers(0, ctx + 1, B)
    new = np.where(rng.random(B) < waits, 0, rng.integers(1, tq + 1, B)) if tq > 0 else np.zeros(B, np.int64)
    held, want = -(-have // page), -(-(have + new) // page)
    cols = cols or int(max(1, -(-(ctx + tq) // page)))
    need = int((want - held).sum())
    spare = need + 3 if spare is None else max(0, int(need * spare))
    ids = rng.permutation(int(held.sum()) + spare + 7).astype(np.int32)
    table = np.full((B, cols), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    free = np.full(len(ids), -5, np.int32)
    free[:spare] = ids[at:at + spare]
    return table, have, new, free, spare, int(new.sum())


@pytest.mark.parametrize("page", [64, 256])
@pytest.mark.parametrize("B,ctx,tq", [(1, 0, 1), (1, 63, 2), (1, 1, 20000), (2, 300, 1), (7, 500, 70), (63, 900, 1),
                                      (64, 130, 64), (65, 900, 5), (130, 40, 400), (1000, 700, 1), (1025, 10, 9),
                                      (3000, 70, 3)])
def test_plan(B, ctx, tq, page):
    rng = np.random.default_rng(B + ctx + tq + page)
    for spare in (None, 0.6, 0.0):
        table, have, new, free, count, tokens = problem(rng, B, ctx, tq, page, spare)
        check_plan(table, have, new, free, count, tokens + int(rng.integers(0, 70)), page, inplace=spare is None)
        check_plan(table, have, new, free, count, max(0, tokens - tokens // 3), page)
    check_plan(table, have, None, free, len(free) - 7, B, page)


def test_plan_of_many_requests():
    rng = np.random.default_rng(5)
    table, have, new, free, count, tokens = problem(rng, 65535, 100, 2, 64, 0.7)
    check_plan(table, have, new, free, count, tokens + 1, 64)


def test_plan_of_any_lengths():
    """Negative and huge lengths take no part and shift no one; ids from outside
    give -1; a count outside the pool is taken into it."""
    rng = np.random.default_rng(8)
    table, have, new, free, count, tokens = problem(rng, 200, 300, 5, 64, cols=9)
    have[[3, 50]], new[[3, 70]] = [-1, -MOST - 1], [4, -3]
    have[[90, 91, 92]], new[[91, 120]] = [MOST, MOST, 577], [MOST, 570]
    table[10, 0], table[11, 0], table[12, 0] = -9, len(free), MOST
    for tok in (tokens, tokens + 4000, 5, 0):
        check_plan(table, have, new, free, count, tok, 64)
    for c in (-5, MOST, len(free) + 1):
        check_plan(table, have, new, np.abs(free), c, tokens + 4000, 64)
    new[100:] = MOST                     # sums past 32 bits
    check_plan(table, have, new, free, count, tokens, 64)
    have[:] = 0
    check_plan(table, have, new, free, count, tokens, 64)
    bad = free.copy()
    bad[:count] = -3
    check_plan(table, have, np.ones(200, int), bad, count, 200, 64)


@pytest.mark.parametrize("B,cols,pages,tokens", [(0, 0, 0, 0), (0, 4, 9, 100), (3, 0, 5, 7), (3, 2, 0, 7), (3, 2, 5, 0)])
def test_plan_of_nothing(B, cols, pages, tokens):
    table = np.zeros((B, cols), np.int32)
    check_plan(table, np.zeros(B, int), np.ones(B, int), np.arange(pages, dtype=np.int32), pages, tokens, 64)


def check_trim(table, held, kept, free, count, page, inplace=False):
    want, left = step_ref.trim(table, held, kept, free, count, page)
    f, buf = guarded(len(free))
    f.copy_(dev(free))
    t, c = dev(table), dev([count])
    got = q.kv_trim(t, dev(held), dev(kept), f, c, page_size=page, left=c if inplace else None)
    assert np.array_equal(f.cpu().numpy(), want) and int(got[0]) == left and intact(buf)
    assert np.array_equal(t.cpu().numpy(), table) and (inplace or int(c[0]) == count)


@pytest.mark.parametrize("B,ctx,cut", [(1, 1, 1), (1, 64, 1), (1, 100000, 100000), (5, 700, 70), (64, 900, 900),
                                       (1000, 300, 64), (1025, 900, 400), (4000, 100, 100)])
def test_trim(B, ctx, cut):
    rng = np.random.default_rng(B + ctx)
    table, have, _, free, count, _ = problem(rng, B, ctx, 0, 64)
    kept = have - rng.integers(0, cut + 1, B)
    for inplace in (False, True):
        check_trim(table, have, kept, free, count, 64, inplace)
        check_trim(table, have, np.zeros(B, int), free, count, 64, inplace)
    check_trim(table, kept, have, free, count, 64)                      # nothing to give back
    check_trim(table, have, np.full(B, -7), free, len(free) - 3, 64)    # the pool has no room: nothing goes back
    check_trim(table, np.full(B, MOST), kept, free, 0, 64)              # held past the columns
    check_trim(table, np.full(B, -MOST - 1), kept, free, -4, 64)
    check_trim(table, have, np.full(B, MOST), free, count, 64)


@pytest.mark.parametrize("B,cols,pages", [(0, 0, 0), (0, 3, 5), (3, 0, 5), (3, 2, 0)])
def test_trim_of_nothing(B, cols, pages):
    check_trim(np.zeros((B, cols), np.int32), np.full(B, 100), np.zeros(B, int), np.zeros(pages, np.int32), 0, 64)


def test_trim_undoes_plan():
    rng = np.random.default_rng(3)
    table, have, new, free, count, tokens = problem(rng, 300, 500, 200, 64, 0.8)
    tab, (_, _, _, granted, left) = check_plan(table, have, new, free, count, tokens, 64)
    f = dev(free)
    after = dev(have) + dev(new) * granted
    back = q.kv_trim(tab, after, dev(have), f, left)
    assert int(back[0]) == count and np.array_equal(f.cpu().numpy(), free) and int(left[0]) < count


def test_outputs_at_any_word():
    """slots and pos that are not 16-byte aligned, rows that are not in fours."""
    rng = np.random.default_rng(12)
    for B, tq, tokens in ((5, 900, 4000), (70, 200, 9001), (3, 40, 50)):
        table, have, new, free, count, _ = problem(rng, B, 300, tq, 64, waits=0.0)
        want = step_ref.plan(table, have, new, free, count, tokens, 64)
        for s_at, p_at in ((1, 0), (0, 3), (2, 1)):
            bufs = [torch.full((tokens + 8,), 77, dtype=torch.int32, device=DEV) for _ in range(2)]
            slots, pos = bufs[0][s_at:s_at + tokens], bufs[1][p_at:p_at + tokens]
            rest = [torch.empty(n, dtype=torch.int32, device=DEV) for n in (B + 1, B, 1)]
            q.kv_plan(dev(table), dev(have), dev(new), dev(free), dev([count]), tokens, out=(rest[0], slots, pos, *rest[1:]))
            assert np.array_equal(slots.cpu().numpy(), want[2]) and np.array_equal(pos.cpu().numpy(), want[3])
            for b, at in zip(bufs, (s_at, p_at)):
                b = b.cpu()
                assert bool((b[:at] == 77).all()) and bool((b[at + tokens:] == 77).all())
