"""Adapters of many requests (lora) against the definition in 64 bits.

Bars, with M the sum of the products' magnitudes and H the row's largest inner
sum times sum |b|: a chain of fp32 sums adds one product or one matrix
instruction's sum at a time, k / 4 of them at most on either side of a join, so
the inner sums are off by (k / 4 + 16) 2^-24 M, the second product by rank 2^-24
(M + H); the two fp16 parts of an inner sum lose 2^-22 H."""
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


class Case:
    def __init__(self, seed, lens, k, outs, rank, n_ad, dtype=F32, gap=0, ranks=None, scale=True, none=True, extra=0):
        gen = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.lens, T = lens, sum(lens) + extra
        self.qstart = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        self.x = torch.randn(T, k + gap, generator=gen).to(dtype)[:, :k]
        self.a = [(torch.randn(n_ad, rank, k, generator=gen) / k ** 0.5).half() for _ in outs]
        self.b = [torch.randn(n_ad, n, rank, generator=gen).half() for n in outs]
        self.base = [torch.randn(T, n, generator=gen) for n in outs]
        self.adapter = rng.integers(-2 if none else 0, n_ad + (1 if none else 0), len(lens)).astype(np.int32)
        self.scale = (torch.rand(n_ad, generator=gen) * 2 - 0.5) if scale else None
        self.ranks = ranks

    def run(self, inplace=True, qstart=True, workspace=None):
        d = lambda t: None if t is None else t.to(DEV)  # noqa: E731
        x = d(self.x.contiguous())
        if self.x.stride(0) != self.x.shape[1]:
            wide = torch.zeros(self.x.shape[0], self.x.stride(0), dtype=self.x.dtype, device=DEV)
            wide[:, :self.x.shape[1]] = x
            wide[:, self.x.shape[1]:] = float("nan")
            x = wide[:, :self.x.shape[1]]
        bufs = [torch.full((b.numel() + 32,), 5.0, device=DEV) for b in self.base]
        ys = [u[16:-16].view(b.shape) for u, b in zip(bufs, self.base)]
        bases = [d(b) for b in self.base]
        if inplace:
            for y, b in zip(ys, bases):
                y.copy_(b)
        tg = [(d(a), d(b), y) if inplace else (d(a), d(b), y, base)
              for a, b, y, base in zip(self.a, self.b, ys, bases)]
        q.lora(x, tg, torch.from_numpy(self.adapter).to(DEV),
               qstart=torch.from_numpy(self.qstart).to(DEV) if qstart else None, scale=d(self.scale),
               ranks=None if self.ranks is None else torch.tensor(self.ranks, dtype=torch.int32, device=DEV),
               workspace=workspace)
        torch.cuda.synchronize()
        for u in bufs:
            assert bool((u[:16] == 5).all()) and bool((u[-16:] == 5).all())
        return ys

    def check(self, ys, untouched=5.0, inplace=True):
        k, rank = self.x.shape[1], self.a[0].shape[1] if self.a else 0
        T = self.qstart[-1]
        want = step_ref.lora(self.x.numpy(), self.adapter, self.qstart,
                             [(a.numpy(), b.numpy(), base.numpy()) for a, b, base in zip(self.a, self.b, self.base)],
                             None if self.scale is None else self.scale.numpy(), self.ranks)
        for y, (w, mag, top), base in zip(ys, want, self.base):
            y = y.cpu().numpy().astype(np.float64)
            bar = ((k / 4 + 16 + rank) * U) * mag + (rank * U + 2.0 ** -22) * top + 4 * U * (np.abs(base.numpy()) + np.abs(w))
            assert np.all(np.abs(y[:T] - w[:T]) <= bar[:T])
            # rows of no request, and of requests without an adapter
            assert np.all(y[T:] == (base.numpy()[T:] if inplace else untouched))
            for i, ad in enumerate(self.adapter):
                if ad < 0 or ad >= self.a[0].shape[0]:
                    rows = slice(self.qstart[i], self.qstart[i + 1])
                    assert np.array_equal(y[rows], base.numpy()[rows].astype(np.float64))


@pytest.mark.parametrize("dtype", [F32, F16])
@pytest.mark.parametrize("lens,k,outs,rank,n_ad", [
    ([1], 8, [1], 8, 1), ([1], 4096, [4096, 1024], 16, 3), ([1] * 5, 64, [7], 8, 2), ([1] * 53, 512, [300, 65], 64, 9),
    ([3], 72, [100], 24, 2), ([17, 1, 40], 136, [33, 4, 129], 32, 3), ([0, 5, 0, 0, 16, 1, 0], 256, [64], 40, 4),
    ([200], 1024, [512], 128, 2), ([15, 16, 17, 31, 33, 1], 4000, [257], 16, 5), ([64, 65, 1, 1, 130], 2048, [1000, 31], 256, 3),
    ([1] * 130, 256, [64], 8, 200), ([2] * 66, 128, [16] * 8, 16, 4), ([1000, 3, 500], 320, [48], 56, 2)])
def test_lora(lens, k, outs, rank, n_ad, dtype):
    c = Case(len(lens) + k, lens, k, outs, rank, n_ad, dtype, gap=8 if k % 16 else 0, extra=3)
    c.check(c.run())
    c.check(c.run(inplace=False), inplace=False)


def test_ranks_hide_what_lies_past_them():
    rng = np.random.default_rng(2)
    ranks = [0, 1, 7, 8, 9, 20, 33, 40, 99, -4]
    for dtype, lens in ((F32, [1] * 30), (F16, [5, 40, 1, 1, 17] * 3), (F32, [70, 3] * 4)):
        c = Case(5, lens, 96, [50, 9], 40, len(ranks), dtype, ranks=ranks, none=False)
        for a, b in zip(c.a, c.b):
            for i, r in enumerate(ranks):
                r = max(0, min(r, 40))
                a[i, r:] = float("nan")
                b[i, :, r:] = float("inf") if rng.random() < 0.5 else float("nan")
        ys = c.run()
        for a, b in zip(c.a, c.b):
            a.nan_to_num_(0, 0, 0)
            b.nan_to_num_(0, 0, 0)
        c.check(ys)


def test_equal_shares_without_starts():
    c = Case(1, [4] * 6, 64, [40], 16, 3, none=False)
    c.check(c.run(qstart=False))


def test_neighbours_do_not_meet():
    """A row with NaN, infinities and huge values leaves every other row's bits as
    they are, in its request's tile and outside."""
    for dtype, lens in ((F32, [9, 1, 1, 30]), (F16, [9, 1, 1, 30]), (F32, [1] * 41)):
        c = Case(3, lens, 128, [70], 16, 2, dtype, none=False)
        good = c.run()[0]
        c.x[4], c.x[10, 3], c.x[20, 5] = float("nan"), float("inf"), 60000.0
        bad = c.run()[0]
        rest = [i for i in range(41) if i not in (4, 10, 20)]
        assert torch.equal(good[rest], bad[rest])
        assert torch.isnan(bad[4]).all() and torch.isfinite(bad[20]).all()


def test_scales_and_magnitudes():
    """Inner sums of any size: their two parts have a common power of two."""
    for s in (1e-12, 1e-4, 1e6, 1e15):
        c = Case(4, [1, 20, 3], 64, [40], 16, 2, scale=False, none=False)
        c.x *= s
        c.base = [b * 0 for b in c.base]
        c.check(c.run())
    c = Case(4, [20], 64, [40], 16, 2, none=False)
    c.x *= 0
    c.check(c.run())


def test_no_adapters_and_nothing():
    c = Case(7, [3, 2], 64, [40], 16, 0, scale=False)
    c.adapter[:] = 0
    c.check(c.run())
    c.check(c.run(inplace=False), inplace=False)
    x = torch.empty(0, 64, device=DEV)
    a, b = torch.zeros(1, 8, 64, dtype=F16, device=DEV), torch.zeros(1, 3, 8, dtype=F16, device=DEV)
    q.lora(x, [(a, b, torch.empty(0, 3, device=DEV))], torch.empty(0, dtype=torch.int32, device=DEV))
    q.lora(torch.empty(2, 64, device=DEV), [], torch.zeros(1, dtype=torch.int32, device=DEV))


def test_the_same_call_gives_the_same_bits():
    c = Case(9, [1] * 20 + [100], 1024, [512, 100], 32, 3)
    first = c.run()
    for _ in range(2):
        assert all(torch.equal(x, y) for x, y in zip(first, c.run()))


def test_starts_from_outside_touch_nothing():
    """Row starts past the tokens, or decreasing: no row outside the buffers is
    read or written."""
    c = Case(2, [4, 4, 4, 4], 64, [40], 16, 2, none=False)
    for starts in ([0, 4, 900, 1000, 2 ** 31 - 1], [-50, 4, 8, 12, 16], [0, 12, 4, 16, 2], [16] * 5, [-9] * 5):
        c.qstart = np.array(starts, np.int32)
        c.run()


@pytest.mark.parametrize("dtype", [F32, F16])
@pytest.mark.parametrize("lens,n_ad", [([1] * 64, 1), ([1] * 150, 2), ([1] * 40, 3), ([1, 1, 30, 1, 0, 1, 1, 2, 1] * 9, 2),
                                       ([1] * 17 + [0] * 200 + [1] * 60, 1), ([1] * 6000, 3)])
def test_equal_adapters_of_single_rows(lens, n_ad, dtype):
    """They share tiles, up to 16 of 64 neighbours, whatever lies between."""
    c = Case(len(lens), lens, 72, [33], 24, n_ad, dtype, extra=2)
    c.check(c.run())
    c.adapter[::3] = -1
    c.check(c.run(inplace=False), inplace=False)


def test_long_requests_end_inside_tiles():
    """64 rows a tile where requests are long on average, beside short and empty ones."""
    for dtype in (F32, F16):
        for rank, outs in ((8, [5]), (24, [700, 33]), (72, [64, 130]), (256, [70])):
            c = Case(rank, [63, 64, 65, 1, 0, 129, 200], 328, outs, rank, 3, dtype, extra=1)
            c.check(c.run())
            c.check(c.run(inplace=False), inplace=False)


@pytest.mark.parametrize("dtype", [F32, F16])
@pytest.mark.parametrize("lens", [[1], [1, 1], [1, 1, 1, 1], [0, 1, 0, 2], [2, 0, 0, 0, 1], [0, 4, 0, 0]])
@pytest.mark.parametrize("k,rank,outs", [(8, 8, [1]), (520, 24, [1025, 7]), (1000, 40, [64, 2100]), (4096, 16, [4096]),
                                         (2048, 64, [300, 1, 33]), (3096, 32, [70])])
def test_the_smallest_calls(k, rank, outs, lens, dtype):
    """One launch where as many requests as tokens bring up to four."""
    for n_ad in (1, 3):
        c = Case(k + rank + n_ad, lens, k, outs, rank, n_ad, dtype, extra=0,
                 ranks=None if n_ad == 1 else [rank - 3, 0, 5])
        c.check(c.run())
        c.check(c.run(inplace=False), inplace=False)
    c.adapter[:] = 0
    for a, b in zip(c.a, c.b):
        a[0, rank - 3:], b[0, :, rank - 3:] = float("nan"), float("inf")
    ys = c.run()
    for a, b in zip(c.a, c.b):
        a.nan_to_num_(0, 0, 0)
        b.nan_to_num_(0, 0, 0)
    c.check(ys)
