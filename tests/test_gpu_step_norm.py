"""rms_norm against the definition in 64 bits.

Bars: a lane adds at most 64 squares in a row, then its waves' sums meet, so the
mean is off by less than 80 roundings of 2^-24, its root by half of that, and the
result by four more: 48 2^-24 of itself, plus half a step of its type."""
import numpy as np
import pytest

import step_ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import dequant_matmul_amd as q  # noqa: E402

DEV = "cuda:0"
U = 2.0 ** -24
F32, F16 = torch.float32, torch.float16
BAR = 48 * U


def half_step(dtype):
    return (0.0, 0.0) if dtype is F32 else (2.0 ** -11, 2.0 ** -25)     # relative, of the smallest fp16 numbers


def values(gen, rows, width, stride, dtype, scale=1.0, offset=0):
    """A [rows, width] view, `stride` between rows, `offset` elements into its buffer."""
    buf = torch.randn(rows * stride + offset + 8, generator=gen) * scale
    return buf.to(dtype).to(DEV)[offset:offset + rows * stride].view(rows, stride)[:, :width]


def near(got, want, dtype):
    rel, least = half_step(dtype)
    got, want = got.double().cpu().numpy(), np.asarray(want)
    assert np.all(np.abs(got - want) <= (BAR + rel) * np.abs(want) + least)


def check(x, res, w, eps, dtype, heads=1):
    rows = x.cpu().numpy().reshape(x.shape[0], heads, -1)
    rr = None if res is None else res.cpu().numpy().reshape(rows.shape)
    s, y = step_ref.norm(rows, rr, None if w is None else w.cpu().numpy(), eps)
    view = x if heads == 1 else x.unflatten(1, (heads, -1))
    rv = res if res is None or heads == 1 else res.unflatten(1, (heads, -1))
    got = q.rms_norm(view, w, residual=rv, eps=eps, dtype=dtype)
    if res is not None:
        got, total = got
        rel, least = half_step(res.dtype)
        assert total.dtype is res.dtype and total.shape == view.shape
        err = np.abs(total.double().cpu().numpy().reshape(s.shape) - s)
        assert np.all(err <= (rel + 2 * U) * np.abs(s) + least)
    assert got.dtype is dtype and got.shape == view.shape
    near(got.reshape(s.shape), y, dtype)


@pytest.mark.parametrize("out", [F32, F16])
@pytest.mark.parametrize("kind", [(F32, None), (F32, F32), (F32, F16), (F16, None), (F16, F16), (F16, F32)])
@pytest.mark.parametrize("T,D,gap", [(1, 8, 0), (3, 1, 0), (5, 7, 1), (2, 64, 0), (4, 100, 12), (17, 513, 3),
                                     (1, 4096, 0), (9, 2048, 64), (3, 1001, 0), (2, 5632, 8), (1, 16384, 0),
                                     (2, 40000, 0), (1, 65536, 0), (1, 65533, 0)])
def test_norm(T, D, gap, kind, out):
    gen = torch.Generator().manual_seed(T * D + gap)
    x = values(gen, T, D, D + gap, kind[0])
    res = None if kind[1] is None else values(gen, T, D, D + 2 * gap, kind[1], 3.0)
    w = (1 + 0.3 * torch.randn(D, generator=gen)).to(DEV)
    check(x, res, w, 1e-5, out)
    check(x, res, None, 1e-6, out)


@pytest.mark.parametrize("dtype", [F32, F16])
@pytest.mark.parametrize("T,H,D,gap", [(1, 32, 128, 0), (7, 8, 64, 24), (300, 4, 80, 160), (33, 14, 64, 0), (5, 3, 8, 8),
                                       (5, 3, 1, 1), (9, 5, 37, 2), (2, 2, 256, 0), (3, 2, 520, 0), (700, 32, 128, 2048)])
def test_norm_of_heads(T, H, D, gap, dtype):
    gen = torch.Generator().manual_seed(T + H + D)
    x = values(gen, T, H * D, H * D + gap, dtype)
    w = (1 + 0.3 * torch.randn(D, generator=gen)).to(DEV)
    check(x, None, w, 1e-6, dtype, heads=H)
    check(x, values(gen, T, H * D, H * D, dtype), w, 1e-6, dtype, heads=H)


@pytest.mark.parametrize("offset", [1, 2, 3, 4])
def test_norm_of_unaligned_rows(offset):
    gen = torch.Generator().manual_seed(offset)
    w = torch.randn(264 + offset, generator=gen).to(DEV)[offset:]
    x, r = values(gen, 5, 264, 264, F32, 1.0, offset), values(gen, 5, 264, 264, F16, 1.0, offset)
    check(x, r, w[:264], 1e-5, F16)
    check(r, x, w[:264], 1e-5, F32)


def test_norm_of_many_rows():
    gen = torch.Generator().manual_seed(2)
    x = torch.randn(70001, 64, generator=gen).half().to(DEV)
    check(x, None, None, 1e-5, F16)
    big = torch.randn(1200, 4096, generator=gen).to(DEV)
    check(big, big.half(), torch.ones(4096, device=DEV), 1e-5, F32)


def test_in_place():
    gen = torch.Generator().manual_seed(4)
    for T, D in ((6, 4096), (40, 96), (3, 1001)):
        x, r = torch.randn(T, D, generator=gen).to(DEV), torch.randn(T, D, generator=gen).to(DEV)
        y, s = q.rms_norm(x, residual=r)
        a, b = x.clone(), r.clone()
        y1, s1 = q.rms_norm(a, residual=b, sum_out=b, out=a)            # both in place
        assert s1 is b and y1 is a and torch.equal(a, y) and torch.equal(b, s)
        a, b = x.clone(), r.clone()
        y2, s2 = q.rms_norm(a, residual=b, sum_out=a, out=b)
        assert torch.equal(s2, s) and torch.equal(y2, y)
        c = x.clone()
        assert torch.equal(q.rms_norm(c, out=c), q.rms_norm(x))


def q8_check(got, y):
    """Blocks against the results in 64 bits: the code of the fp32 result, whose place
    on the code's scale is off by no more than 127 times twice its bar, rounds to a
    whole number at most 1/2 away; the scale is fp16."""
    blk = got.cpu().numpy().reshape(-1, 34)
    y = y.reshape(-1, 32)
    d = np.abs(y).max(-1) / 127
    d16 = blk[:, :2].copy().view(np.float16)[:, 0].astype(np.float64)
    assert np.all(np.abs(d16 - d) <= (2.0 ** -11 + BAR + 2 * U) * d + 2.0 ** -25)
    code = blk[:, 2:].view(np.int8).astype(np.float64)
    at = y / np.where(d > 0, d, 1)[:, None]
    assert np.all(np.abs(code - at) <= 0.5 + 127 * (2 * BAR + 4 * U))
    assert np.all(np.abs(code).max(-1)[d > 0] == 127) and np.all(code[d == 0] == 0)


@pytest.mark.parametrize("kind", [(F32, None), (F32, F32), (F16, F16), (F16, F32), (F32, F16)])
@pytest.mark.parametrize("T,H,D", [(1, 1, 4096), (1, 1, 32), (5, 1, 96), (3, 1, 5632), (2, 1, 14336), (1, 1, 65536),
                                   (41, 1, 2080), (6, 8, 64), (3, 3, 96), (700, 1, 512)])
def test_q8_blocks(T, H, D, kind):
    gen = torch.Generator().manual_seed(T + D)
    x = values(gen, T, H * D, H * D + 8, kind[0])
    res = None if kind[1] is None else values(gen, T, H * D, H * D, kind[1])
    w = (1 + 0.3 * torch.randn(D, generator=gen)).to(DEV)
    s, y = step_ref.norm(x.cpu().numpy().reshape(T, H, D), None if res is None else res.cpu().numpy().reshape(T, H, D),
                         w.cpu().numpy(), 1e-5)
    buf = torch.full((T * q.row_bytes(q.Q8_0, H * D) + 64,), 77, dtype=torch.uint8, device=DEV)
    out = buf[32:-32].view(T, -1)
    args = [t if t is None or H == 1 else t.unflatten(1, (H, D)) for t in (x, res)]
    got = q.rms_norm(args[0], w, residual=args[1], eps=1e-5, qtype=q.Q8_0, out=out)
    got, total = (got, None) if res is None else got
    assert got is out and bool((buf[:32] == 77).all()) and bool((buf[-32:] == 77).all())
    q8_check(got, y)
    if total is not None:
        assert np.all(np.abs(total.double().cpu().numpy().reshape(s.shape) - s)
                      <= (half_step(res.dtype)[0] + 2 * U) * np.abs(s) + 2.0 ** -25)


def test_q8_is_the_quantizer_of_the_fp32_norm():
    gen = torch.Generator().manual_seed(6)
    for T, D in ((3, 4096), (65, 224)):
        x, w = torch.randn(T, D, generator=gen).to(DEV), torch.randn(D, generator=gen).to(DEV)
        assert torch.equal(q.rms_norm(x, w, qtype=q.Q8_0), q.quantize(q.rms_norm(x, w), q.Q8_0))


def test_special_values():
    x = torch.zeros(6, 96, device=DEV)
    x[1, 5], x[2, 6], x[3], x[5] = float("nan"), float("inf"), 1e-30, -2.0
    y = q.rms_norm(x, eps=1e-5)
    assert torch.equal(y[0], torch.zeros(96, device=DEV)) and torch.isnan(y[1]).all()
    assert torch.isnan(y[2, 6]) and (y[2, :6] == 0).all() and torch.isfinite(y[3]).all()
    assert (y[4] == 0).all() and torch.allclose(y[5], torch.full((96,), -1.0, device=DEV), rtol=1e-5)
    half = q.rms_norm(torch.ones(1, 32, device=DEV), torch.full((32,), 1e6, device=DEV), dtype=F16)
    assert torch.isinf(half).all()
    b = q.rms_norm(x[:1], qtype=q.Q8_0).cpu().numpy().reshape(-1, 34)
    assert not b.any()                                             # a zero row: zero codes and scales
    # a row whose squares are too small for fp32 is governed by eps
    t = torch.full((1, 64), 1e-25, device=DEV)
    assert torch.allclose(q.rms_norm(t, eps=1e-6), t * 1e3, rtol=1e-6)


def test_empty():
    assert q.rms_norm(torch.empty(0, 64, device=DEV)).shape == (0, 64)
    assert q.rms_norm(torch.empty(3, 0, device=DEV)).shape == (3, 0)
    assert q.rms_norm(torch.empty(3, 0, 8, device=DEV)).shape == (3, 0, 8)
