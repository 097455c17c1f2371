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
