"""kv_plan where lengths and pages come near 2^31 tokens, against the definition in
whole numbers."""
import numpy as np
import pytest

import step_ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import dequant_matmul_amd as q  # noqa: E402

DEV = "cuda:0"
I32 = torch.int32


@pytest.fixture(autouse=True)
def released():
    yield
    torch.cuda.empty_cache()


def dev(v):
    return torch.tensor(v, dtype=I32, device=DEV)


@pytest.mark.parametrize("page,ctx,fresh", [
    (1 << 30, [(1 << 30) + 5, 7], [100, 3]), (1 << 30, [(1 << 30) + 5, 7], [100, 5000]),
    (1 << 30, [2 ** 31 - 12, 0], [11, 600]), (1 << 24, [2 ** 31 - 3000, 2 ** 31 - 2 ** 23], [2999, 20]),
    (1 << 20, [2 ** 31 - 2 ** 19, 5], [7000, 9])])
def test_rows_of_the_last_page_of_the_largest_contexts(page, ctx, fresh):
    """The old page that has room is the last one below 2^31 tokens."""
    cols, pages = 2 ** 31 // page, min(2 ** 31 // page - 1, 40)
    table = np.full((2, cols), 0, np.int32)
    pool, tokens = np.arange(pages, dtype=np.int32)[::-1].copy(), sum(fresh) + 3
    want = step_ref.plan(table, ctx, fresh, pool, pages, tokens, page)
    t, free, count = dev(table), dev(pool), dev([pages])
    qstart, slots, pos, granted, left = q.kv_plan(t, dev(ctx), dev(fresh), free, count, tokens, page_size=page)
    got = (t, qstart, slots, pos, granted)
    for g, w in zip(got, want):
        assert np.array_equal(g.cpu().numpy(), w)
    assert int(left[0]) == want[5]


def test_rows_of_the_last_small_page():
    """Pages of 64 up to 2^31 - 1 tokens."""
    cols = 2 ** 31 // 64
    table = torch.zeros(1, cols, dtype=I32, device=DEV)
    table[0, -1] = 3
    c, n = 2 ** 31 - 40, 39
    free, count = dev([5, 6, 7, 8]), dev([2])
    _, slots, pos, granted, left = q.kv_plan(table, dev([c]), dev([n]), free, count, n)
    assert granted.tolist() == [1] and int(left[0]) == 2
    p = np.arange(c, c + n)
    assert slots.tolist() == (3 * 64 + p % 64).tolist() and pos.tolist() == p.tolist()


@pytest.mark.parametrize("lens,wide", [([2 ** 31 - 1] * 4 + [1], False), ([2 ** 30, 2 ** 30, 2 ** 30, 2 ** 30, 64, 0], False),
                                       ([5, 2 ** 31 - 8, 2, 1], True)])
def test_the_most_tokens(lens, wide):
    """tokens = 2^31 - 1, and lengths whose sum is past that: no later request comes out
    at an earlier row.  `wide`: the table's rows hold them all, and nothing is short."""
    T, B = 2 ** 31 - 1, len(lens)
    cols = 2 ** 31 // 2 ** 30 if wide else 4
    page = 2 ** 30 if wide else 64
    pages = 1 if wide else 100
    table = torch.zeros(B, cols, dtype=I32, device=DEV)
    ctx = dev([3 if wide else 0] * B)         # (wide: on their one old page)
    free, count = torch.arange(pages, dtype=I32, device=DEV), dev([pages])
    qstart, slots, pos, granted, left = q.kv_plan(table, ctx, dev(lens), free, count, T, page_size=page)
    starts = [min(sum(lens[:i]), T) for i in range(B + 1)]
    assert qstart.tolist() == starts
    fits = [3 * wide + n <= min(cols * page, T) and sum(lens[:i + 1]) <= T for i, n in enumerate(lens)]
    need = [-(-(3 * wide + n) // page) - wide if f else 0 for n, f in zip(lens, fits)]
    ok = [int(f and (w == 0 or sum(need[:i + 1]) <= pages)) for i, (f, w) in enumerate(zip(fits, need))]
    assert granted.tolist() == ok and int(left[0]) == pages - sum(w for w, o in zip(need, ok) if o)
    for b in range(B):
        lo, hi = starts[b], starts[b + 1]
        if not ok[b] and hi > lo:
            assert int(slots[lo:hi].max()) == -1 and int(pos[lo:hi].max()) == 0
        elif hi > lo:
            assert int(pos[lo]) == 3 * wide and int(pos[hi - 1]) == 3 * wide + hi - lo - 1
            assert int(slots[lo:hi].min()) >= 0
    if starts[-1] < T:
        assert int(slots[starts[-1]:].max()) == -1
