"""rms_norm of rows whose squares pass the largest fp32 number, against the definition
in 64 bits.  Bars as for ordinary rows: 48 roundings of 2^-24 (the power of two that
such a row is brought down by rounds nothing), plus half a step of the result's type."""
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
MOST = 3.4028234663852886e38


def rows(T, D, scale, seed, offset=0):
    """fp32 rows of values up to `scale`, each row's a little smaller than the one before."""
    rng = np.random.default_rng(seed)
    v = rng.uniform(-1, 1, (T, D)) * scale * 0.9 ** np.arange(T)[:, None]
    buf = torch.zeros(T * D + 8, device=DEV)
    x = buf[offset:offset + T * D].view(T, D)
    x.copy_(torch.from_numpy(v.astype(np.float32)))
    return x


@pytest.mark.parametrize("scale", [1e16, 1e18, 3e19, 1e25, 1e33, MOST / 4, MOST])
@pytest.mark.parametrize("T,D,offset", [(1, 1, 0), (3, 8, 0), (5, 64, 0), (9, 128, 0), (2, 200, 0), (3, 512, 0), (2, 4096, 0),
                                        (3, 2048, 0), (2, 8192, 0), (2, 16384, 0), (1, 65536, 0), (3, 77, 0), (2, 1001, 0),
                                        (2, 4096, 1), (1, 65533, 0)])
def test_rows_whose_squares_pass_fp32(T, D, offset, scale):
    x = rows(T, D, scale, T + D, offset)
    w = 1 + 0.3 * torch.randn(D, generator=torch.Generator().manual_seed(D))
    _, want = step_ref.norm(x.cpu().numpy(), None, w.numpy(), 1e-5)
    got = q.rms_norm(x, w.to(DEV), eps=1e-5).double().cpu().numpy()
    assert np.all(np.abs(got - want) <= 48 * U * np.abs(want) + 2.0 ** -140)
    half = q.rms_norm(x, w.to(DEV), eps=1e-5, dtype=F16).double().cpu().numpy()
    assert np.all(np.abs(half - want) <= (48 * U + 2.0 ** -11) * np.abs(want) + 2.0 ** -25)
    if D % 32 == 0:
        y = q.rms_norm(x, w.to(DEV), eps=1e-5)
        assert torch.equal(q.rms_norm(x, w.to(DEV), eps=1e-5, qtype=q.Q8_0), q.quantize(y, q.Q8_0))


@pytest.mark.parametrize("H,D", [(4, 64), (3, 128), (5, 40), (2, 520), (3, 37)])
def test_large_rows_beside_ordinary_ones(H, D):
    """In one wave or workgroup; the ordinary rows' bits are what they are alone, and the
    sum that is stored is not brought down."""
    x = torch.randn(6, H, D, generator=torch.Generator().manual_seed(D))
    res = torch.randn(6, H, D, generator=torch.Generator().manual_seed(D + 1))
    plain = q.rms_norm(x.to(DEV), residual=res.to(DEV))
    big = x.clone()
    big[1::2, 0] *= 1e30
    y, s = q.rms_norm(big.to(DEV), residual=res.to(DEV))
    ws, want = step_ref.norm(big.numpy(), res.numpy(), None, 1e-6)
    assert torch.equal(y[0::2], plain[0][0::2]) and torch.equal(y[:, 1:], plain[0][:, 1:])
    assert np.all(np.abs(s.double().cpu().numpy() - ws) <= U * np.abs(ws))
    # (s enters unrounded to `sum`, of which 2^-24 is lost, too)
    assert np.all(np.abs(y.double().cpu().numpy() - want) <= 50 * U * np.abs(want) + 2.0 ** -140)


def test_eps_of_large_rows():
    """An eps as large as the mean still counts."""
    x = rows(3, 96, 1e19, 2)
    for eps in (1e36, 1e38):
        _, want = step_ref.norm(x.cpu().numpy(), None, None, eps)
        got = q.rms_norm(x * 10, eps=eps).double().cpu().numpy()
        _, want = step_ref.norm((x * 10).cpu().numpy(), None, None, eps)
        assert np.all(np.abs(got - want) <= 48 * U * np.abs(want))


def test_rows_that_are_not_numbers_stay_so():
    x = torch.ones(4, 4096, device=DEV)
    x[0, 7], x[1, 9], x[2] = float("nan"), float("inf"), 3e38
    y = q.rms_norm(x)
    assert torch.isnan(y[0]).all() and torch.isnan(y[1, 9]) and (y[1, :9] == 0).all()
    assert torch.allclose(y[2], torch.ones(4096, device=DEV), rtol=1e-5)
    assert torch.allclose(y[3], torch.ones(4096, device=DEV), rtol=1e-5)
