"""Buffers past 4 GiB: rows, pages and weights whose offsets pass 32 bits are the
right ones (those at the end of the buffers, checked alone)."""
import numpy as np
import pytest

import qmm_inputs as G

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


def test_norm_rows_past_4_gib():
    T, D = 600001, 4096
    x = torch.zeros(T, D, dtype=torch.float16, device=DEV)
    x[-3:] = torch.randn(3, D, device=DEV).half()
    out, total = q.rms_norm(x, residual=x, eps=1e-5)
    want = q.rms_norm(x[-3:].contiguous(), residual=x[-3:].contiguous(), eps=1e-5)
    assert torch.equal(out[-3:], want[0]) and torch.equal(total[-3:], want[1])
    assert not out[:-3].any()
    blocks = q.rms_norm(x, qtype=q.Q8_0)
    assert torch.equal(blocks[-3:], q.rms_norm(x[-3:].contiguous(), qtype=q.Q8_0))


def test_table_entries_past_4_gib():
    B, cols = 3, 1 << 30
    table = torch.full((B, cols), -1, dtype=I32, device=DEV)
    table[2, :3] = torch.tensor([7, 8, 9], dtype=I32, device=DEV)
    ctx, fresh = torch.tensor([0, 5, 150], dtype=I32, device=DEV), torch.tensor([1, 0, 200], dtype=I32, device=DEV)
    table[1, 0] = 3
    free, count = torch.arange(100, 200, dtype=I32, device=DEV), torch.tensor([50], dtype=I32, device=DEV)
    free[50:] = 0
    pages = 1000
    pool = torch.zeros(pages, dtype=I32, device=DEV)
    pool[:50] = free[:50]
    qstart, slots, pos, granted, left = q.kv_plan(table, ctx, fresh, pool, count, 201)
    assert granted.tolist() == [1, 1, 1] and int(left[0]) == 46 and qstart.tolist() == [0, 1, 1, 201]
    assert table[0, 0] == 149 and table[2, :7].tolist() == [7, 8, 9, 148, 147, 146, -1]
    p = np.arange(150, 350)
    row = np.array([7, 8, 9, 148, 147, 146])
    assert slots.tolist() == [149 * 64] + (row[p // 64] * 64 + p % 64).tolist()
    held = torch.tensor([0, 0, 350], dtype=I32, device=DEV)
    back = q.kv_trim(table, held, torch.tensor([0, 0, 150], dtype=I32, device=DEV), pool, left)
    assert int(back[0]) == 49 and pool[46:49].tolist() == [146, 147, 148]


def test_weights_past_4_gib():
    k, n = 4096, 1100001
    rb = q.row_bytes(q.Q8_0, k)
    w = torch.zeros(n * rb, dtype=torch.uint8, device=DEV)
    tail = torch.from_numpy(G.gen_weights(G.Q8_0, 40, k, 5).reshape(-1)).to(DEV)
    w[-tail.numel():] = tail
    for batch in (1, 5):
        x = q.quantize(torch.randn(batch, k, device=DEV), q.Q8_0)
        y = q.gemv_q8(w, q.Q8_0, n, k, x)
        assert torch.equal(y[:, -40:], q.gemv_q8(tail, q.Q8_0, 40, k, x)) and not y[:, :-40].any()


@pytest.mark.parametrize("lens", [[1] * 3 + [40], [16000, 16000, 20000, 4000]])
def test_adapters_past_4_gib(lens):
    """The last of many adapters, and outputs of many rows."""
    T, k, n, rank = sum(lens), 64, 30000, 16
    n_ad = 4500
    a = torch.zeros(n_ad, rank, k, dtype=torch.float16, device=DEV)
    b = torch.zeros(n_ad, n, rank, dtype=torch.float16, device=DEV)
    a[-1], b[-1] = torch.randn(rank, k, device=DEV).half(), torch.randn(n, rank, device=DEV).half()
    x, y = torch.randn(T, k, device=DEV).half(), torch.zeros(T, n, device=DEV)
    pick = torch.full((len(lens),), n_ad - 1, dtype=I32, device=DEV)
    starts = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=I32, device=DEV)
    q.lora(x, [(a, b, y)], pick, qstart=starts)
    for rows in (slice(0, 5), slice(T - 20, T)):
        want = (x[rows].double() @ a[-1].double().T) @ b[-1].double().T
        bar = (x[rows].double().abs() @ a[-1].double().abs().T) @ b[-1].double().abs().T
        assert bool(((y[rows].double() - want).abs() <= 100 * 2.0 ** -24 * bar).all())


def test_adapters_of_the_widest_targets():
    """More blocks of columns than a grid's second dimension takes."""
    n, k, rank = 1 << 24, 8, 8
    a, b = torch.randn(1, rank, k, device=DEV).half(), torch.zeros(1, n, rank, dtype=torch.float16, device=DEV)
    b[0, -5:], b[0, :5] = 1.0, 2.0
    x = torch.randn(3, k, device=DEV)
    ys = [torch.zeros(3, n, device=DEV) for _ in range(8)]
    q.lora(x, [(a, b, y) for y in ys], torch.zeros(3, dtype=I32, device=DEV))
    h = (x.double() @ a[0].double().T).sum(-1)
    for y in ys:
        assert bool(((y[:, -5:].double() - h[:, None]).abs() < 1e-4).all())
        assert bool(((y[:, :5].double() - 2 * h[:, None]).abs() < 1e-4).all()) and not y[:, 5:-5].any()
