"""Rotation and append of more tokens than the work-items of one launch (2^32) reach.

Tokens are told apart by small whole numbers, exact in fp16, and turned by a quarter:
(a, b) becomes (-b, a) whatever the order of rounding."""
import pytest

import kv_ref as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import dequant_matmul_amd as q  # noqa: E402

DEV = "cuda:0"


def test_rope_of_more_tokens_than_a_launch():
    """One pair of 136 dims in the half layout: a workgroup a token."""
    T = (1 << 24) + 5
    x = torch.empty(T, 1, 136, dtype=torch.float16, device=DEV)
    t = torch.arange(T, device=DEV)
    x[:, 0, 0], x[:, 0, 1], x[:, 0, 2:] = (t % 2039).half(), (t % 2029).half(), 3.0
    cs = torch.zeros(T, 1, 2, device=DEV)
    cs[..., 1] = 1
    q.rope(x, cs, out=x)
    assert torch.equal(x[:, 0, 0], -(t % 2029).half()) and torch.equal(x[:, 0, 1], (t % 2039).half())
    assert (x[:, 0, 2:] == 3).all()


@pytest.mark.parametrize("rotated", [False, True])
def test_append_of_more_tokens_than_a_launch(rotated):
    """8-wide heads: a workgroup takes 64 tokens.  All but three hundred are padding."""
    T, L = (1 << 30) + 70, 300
    kv = torch.empty(T, 1, 8, dtype=torch.float16, device=DEV)
    slots = torch.full((T,), -1, dtype=torch.int32, device=DEV)
    at = torch.cat([torch.arange(100), (1 << 29) - 50 + torch.arange(100), T - 100 + torch.arange(100)]).to(DEV)
    slots[at] = torch.arange(L, dtype=torch.int32, device=DEV)
    rows = torch.arange(L * 8, device=DEV).reshape(L, 1, 8) % 2039
    kv[at] = rows.half()
    cs = None
    if rotated:
        cs = torch.zeros(T, 1, 2, device=DEV)
        cs[at, :, 1] = 1
    cache = q.KVCache(R.F16, 1, 8, 5)
    q.kv_append(cache, kv, kv, slots, cs=cs)
    k, v = q.kv_read(cache, torch.arange(L, dtype=torch.int32, device=DEV))
    assert torch.equal(v, rows.float())
    if rotated:
        rows = torch.cat([-rows[..., 1:2], rows[..., :1], rows[..., 2:]], -1)
    assert torch.equal(k, rows.float())


@pytest.mark.parametrize("kind", ["f16", "q8_0"])
def test_read_and_move_of_more_rows_than_a_launch(kind):
    """65535 workgroups of 16 rows, of one group: every slot of a cache read in a
    shuffled order, then moved one by one from its lower to its upper half."""
    half = 1 << 20
    gen = torch.Generator(device=DEV).manual_seed(1)
    cache = q.KVCache(R.TYPES[kind], 1, 8, 2 * half // 256, page_size=256)
    rows = torch.randint(-100, 100, (half, 1, 8), device=DEV, generator=gen)
    rows[..., 0] = 127              # the scale of a Q8_0 block is 1
    every = torch.arange(half, dtype=torch.int32, device=DEV)
    q.kv_append(cache, rows.half(), -rows.half(), every)
    order = torch.randperm(half, device=DEV, generator=gen)
    order = torch.cat([order, order[:70]])
    k, v = q.kv_read(cache, order.int())
    assert torch.equal(k, rows[order].float()) and torch.equal(v, -rows[order].float())
    q.kv_move(cache, every[:, None].contiguous(), (every + half)[:, None].contiguous())
    k, v = q.kv_read(cache, every + half)
    assert torch.equal(k, rows.float()) and torch.equal(v, -rows.float())
