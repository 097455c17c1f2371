"""Adapters at the C entry's edges: targets without columns, and workspaces of the
least size between guards."""
import ctypes

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import dequant_matmul_amd as q  # noqa: E402
from dequant_matmul_amd import step  # noqa: E402

DEV = "cuda:0"
I32 = torch.int32
F32, F16 = torch.float32, torch.float16


def call(x, targets, adapter, qstart, workspace, rank, n_ad):
    """qst_lora itself: targets are (a, b, base, y, n) with tensors or numbers."""
    at = lambda t: t if t is None or isinstance(t, int) else t.data_ptr()  # noqa: E731
    tab = (step.LoraTarget * len(targets))(*[step.LoraTarget(*[at(v) for v in t[:4]], t[4]) for t in targets])
    a = step.LoraArgs(x.data_ptr(), adapter.data_ptr(), qstart.data_ptr(), None, None, at(workspace),
                      0 if workspace is None else workspace.numel(), x.stride(0), x.shape[0], adapter.numel(),
                      x.shape[1], n_ad, rank, 0 if x.dtype is F32 else 1, len(targets))
    need = q.lib.qst_lora_workspace(ctypes.addressof(a))
    if workspace is None:
        return need
    return q.lib.qst_lora(ctypes.addressof(a), ctypes.addressof(tab), torch.cuda.current_stream().cuda_stream)


@pytest.mark.parametrize("dtype", [F32, F16])
@pytest.mark.parametrize("lens,k,rank", [([1] * 9, 2048, 24), ([1, 1], 264, 16), ([40, 90, 64], 1032, 40),
                                         ([200], 8192, 136)])
@pytest.mark.parametrize("place", [[0], [1], [0, 2], [0, 1, 2, 3, 4, 5, 6]])
def test_targets_without_columns(place, lens, k, rank, dtype):
    """Their pointers may be NULL or of any alignment; the others' results are those of
    a call that is not given them, up to the order of the sums."""
    gen = torch.Generator().manual_seed(k + rank)
    T, n_ad, ns = sum(lens), 2, [70, 33]
    x = torch.randn(T, k, generator=gen).to(dtype).to(DEV)
    a = [(torch.randn(n_ad, rank, k, generator=gen) / k ** 0.5).half().to(DEV) for _ in ns]
    b = [torch.randn(n_ad, n, rank, generator=gen).half().to(DEV) for n in ns]
    ys = [torch.zeros(T, n, device=DEV) for n in ns]
    adapter = torch.tensor([i % 3 - (i % 3 == 2) * 3 for i in range(len(lens))], dtype=I32, device=DEV)
    qstart = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=I32, device=DEV)
    targets = list(zip(a, b, [None, None], ys, ns))
    for i in place:                     # (a NULL a, and one at an odd byte: neither is looked at)
        targets.insert(min(i, len(targets)), (None, None, None, None, 0) if i % 2 == 0 else (1, 3, 5, 7, 0))
    targets = targets[:8]
    guard = 256
    need = call(x, targets, adapter, qstart, None, rank, n_ad)
    buf = torch.full((need + 2 * guard,), 77, dtype=torch.uint8, device=DEV)
    assert call(x, targets, adapter, qstart, buf[guard:guard + need], rank, n_ad) == q.OK
    torch.cuda.synchronize()
    assert bool((buf[:guard] == 77).all()) and bool((buf[guard + need:] == 77).all())
    for u, v, y in zip(a, b, ys):
        if not any(t[3] is y for t in targets):
            continue
        want, bar = torch.zeros_like(y, dtype=torch.float64), torch.ones_like(y, dtype=torch.float64)
        for i, n in enumerate(lens):
            at, rows = int(adapter[i]), slice(int(qstart[i]), int(qstart[i + 1]))
            if at < 0:
                continue
            h, m = x[rows].double() @ u[at].double().T, x[rows].double().abs() @ u[at].double().abs().T
            want[rows] = h @ v[at].double().T
            # (k / 4 + 16 + rank) 2^-24 of the products' magnitudes, 2^-22 and rank 2^-24 of the
            # row's largest inner sum times sum |b|, four roundings of the result
            bar[rows] = ((k / 4 + 16 + rank) * 2.0 ** -24) * (m @ v[at].double().abs().T) \
                + (2.0 ** -22 + rank * 2.0 ** -24) * h.abs().amax(-1, keepdim=True) * v[at].double().abs().sum(-1)[None] \
                + 2.0 ** -22 * want[rows].abs()
            assert bool(((y[rows].double() - want[rows]).abs() <= bar[rows]).all())
        none = torch.cat([torch.full((n,), int(adapter[i]) < 0) for i, n in enumerate(lens)])
        assert not y[none.to(DEV)].any()


@pytest.mark.parametrize("dtype", [F32, F16])
@pytest.mark.parametrize("rank", [8, 40, 136])
@pytest.mark.parametrize("k", [64, 2056])
@pytest.mark.parametrize("starts", [
    [0, 4, 8, 12, 16], [0, 4, 900, 1000, 2 ** 31 - 1], [-50, 4, 8, 12, 16], [0, 12, 4, 16, 2], [16] * 5, [-9] * 5, [0, 16],
    [-2 ** 31, 2 ** 31 - 1], [3, 200], [0, 1, 2, 3, 4], list(range(0, 200, 3)), list(range(0, -200, -3)),
    [0] * 70 + [2 ** 31 - 1] * 60])
def test_workspace_and_outputs_between_guards(starts, k, rank, dtype):
    """Row starts in and out of order, inside and outside of the tokens, with a workspace
    of the least size: nothing around it or the outputs is written."""
    for T in (16, 150):
        gen = torch.Generator().manual_seed(T + k)
        x = torch.randn(T, k, generator=gen).to(dtype).to(DEV)
        n_ad, n = 2, 70
        a = (torch.randn(n_ad, rank, k, generator=gen) / k ** 0.5).half().to(DEV)
        b = torch.randn(n_ad, n, rank, generator=gen).half().to(DEV)
        adapter = torch.arange(len(starts) - 1, dtype=I32, device=DEV) % 3
        qstart = torch.tensor(starts, dtype=I32, device=DEV)
        out = torch.full((T * n + 32,), 5.0, device=DEV)
        y = out[16:-16].view(T, n)
        targets = [(a, b, None, y, n)]
        need = call(x, targets, adapter, qstart, None, rank, n_ad)
        buf = torch.full((need + 512,), 77, dtype=torch.uint8, device=DEV)
        assert call(x, targets, adapter, qstart, buf[256:256 + need], rank, n_ad) == q.OK
        torch.cuda.synchronize()
        assert bool((buf[:256] == 77).all()) and bool((buf[256 + need:] == 77).all())
        assert bool((out[:16] == 5).all()) and bool((out[-16:] == 5).all())
        assert call(x, targets, adapter, qstart, buf[256:256 + need - 16], rank, n_ad) == q.ERR_WORKSPACE
