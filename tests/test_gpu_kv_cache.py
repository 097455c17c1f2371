"""GPU tests of the rotary positions and the paged KV cache: angles, rotation,
append, read back and move, against the definitions of kv_ref.py and the
oracle's encoder.

Bars.  Angles: the fp32 rounding of a 64-bit value, half a step (2^-24) with
the device's 64-bit sine and cosine a few units of 2^-53 off, so 2^-24 + 2^-48 of
a value of magnitude at most 1 (times the factor).  Rotation: two products and a
sum, each rounded to fp32: |error| <= 2^-24 (|a c| + |b s| + |result|) to first
order, and one rounding to the output type.  Cache: the stored values are those
of the oracle's encoder on the same fp32 values, exactly.
"""
import numpy as np
import pytest

import kv_ref as R
import oracle

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import dequant_matmul_amd as q  # noqa: E402

DEV = "cuda:0"


def up(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def normal(rng, *shape, dt=np.float32):
    return rng.standard_normal(shape).astype(np.float32).astype(dt)


@pytest.mark.parametrize("pairs", [1, 16, 33, 64])
def test_angles(pairs):
    rng = np.random.default_rng(pairs)
    pos = np.concatenate([[0, 1, -1, -70000, 1 << 20, (1 << 31) - 1, -(1 << 31)],
                          rng.integers(0, 1 << 20, 60)]).astype(np.int32)
    f, m = q.rope_freqs(2 * pairs, 500000.0, "yarn", factor=16, trained=4096)
    got = q.rope_angles(up(pos), f.to(DEV), m).cpu().numpy()
    ref = R.angles(pos, f.numpy(), m)
    assert np.all(np.abs(got - ref) <= m * (2.0 ** -24 + 2.0 ** -48))
    assert q.rope_angles(up(pos[:0]), f.to(DEV), m).shape == (0, pairs, 2)


ROPES = [(1, 32, 128, 128), (5, 32, 128, 64), (300, 4, 64, 64), (3, 7, 80, 32), (9, 3, 96, 96), (2, 5, 72, 20),
         (4, 2, 40, 14), (33, 1, 8, 2), (17, 3, 256, 0), (7, 2, 64, 48)]


@pytest.mark.parametrize("dt", [np.float32, np.float16])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T,H,D,rot", ROPES)
def test_rope(T, H, D, rot, inter, dt):
    rng = np.random.default_rng(T * 1000 + D + rot)
    pos = rng.integers(0, 100000, T).astype(np.int32)
    cs = R.angles(pos, R.np.power(10000.0, -np.arange(rot // 2) / max(rot // 2, 1)), 1.25).astype(np.float32)
    x = normal(rng, T, H, D, dt=dt)
    ref = R.rotate(x.astype(np.float64), cs.astype(np.float64), inter)
    size = R.rotate(np.abs(x).astype(np.float64), np.abs(cs).astype(np.float64) * [1, -1], inter)   # |a c| + |b s|, one of the pair
    size = np.maximum(np.abs(size), np.abs(ref)) + np.abs(R.rotate(np.abs(x).astype(np.float64), np.abs(cs).astype(np.float64), inter))
    tol = 3 * 2.0 ** -24 * size + (2.0 ** -11 * np.abs(ref) + 2.0 ** -25 if dt == np.float16 else 0)
    xd, cd = up(x), up(cs)
    got = q.rope(xd, cd, interleaved=inter)
    assert np.all(np.abs(got.cpu().numpy() - ref) <= tol)
    assert np.array_equal(got[..., rot:].cpu().numpy(), x[..., rot:])
    # a strided view of a wider projection output, in place: the same bits, the rest untouched
    wide = torch.full((T, H * D + 48), 7.0, dtype=xd.dtype, device=DEV)
    view = wide[:, 16:16 + H * D].unflatten(1, (H, D))
    view.copy_(xd)
    q.rope(view, cd, interleaved=inter, out=view)
    assert torch.equal(view, got)
    assert (wide[:, :16] == 7).all() and (wide[:, 16 + H * D:] == 7).all()


def make(kind, kvh, D, pages, page=64):
    """A cache whose bytes are all ones (NaN where nothing was written)."""
    c = q.KVCache(R.TYPES[kind], kvh, D, pages, page_size=page)
    c.k.fill_(255)
    c.v.fill_(255)
    return c


KINDS = ["f16", "q8_0", "q4_0"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [8, 64, 80, 96, 128, 200, 256])
@pytest.mark.parametrize("dt", [np.float32, np.float16])
def test_append_and_read(kind, D, dt):
    rng = np.random.default_rng(D)
    kvh, page, pages, T = 3, 128, 5, 150
    k, v = (normal(rng, T, kvh, D, dt=dt) for _ in range(2))
    k[3] = 0
    v[5, 1, :] = -2
    v[6, 0, :8] = [3, -3, 0, 0, 1e-3, -1e-3, 2, 1]
    slots = rng.permutation(pages * page)[:T].astype(np.int32)
    slots[:70] = np.arange(70) + 2 * page + 21          # a run from inside a tile
    slots[70:] = rng.permutation(np.setdiff1d(np.arange(pages * page), slots[:70]))[:T - 70]
    c = make(kind, kvh, D, pages, page)
    q.kv_append(c, up(k), up(v), up(slots))
    order = rng.permutation(T)
    gk, gv = q.kv_read(c, up(slots[order]))
    for got, x in ((gk, k), (gv, v)):
        assert np.array_equal(got.cpu().numpy(), R.stored(x.astype(np.float32), kind)[order])
    hk, hv = q.kv_read(c, up(slots[order]), torch.float16)
    assert torch.equal(hk, gk.half()) and torch.equal(hv, gv.half())
    # rows not written keep their bytes: write other rows, read the first again
    rest = np.setdiff1d(np.arange(pages * page), slots).astype(np.int32)[:77]
    k2, v2 = (normal(rng, 77, kvh, D, dt=dt) for _ in range(2))
    q.kv_append(c, up(k2), up(v2), up(rest))
    ak, av = q.kv_read(c, up(slots[order]))
    assert torch.equal(ak, gk) and torch.equal(av, gv)
    # slots outside the cache: nothing written, zeros read
    before = c.k.clone(), c.v.clone()
    bad = np.array([-1, pages * page, (1 << 31) - 1, -(1 << 31)], np.int32)
    q.kv_append(c, up(k[:4]), up(v[:4]), up(bad))
    assert torch.equal(before[0], c.k) and torch.equal(before[1], c.v)
    zk, zv = q.kv_read(c, up(bad))
    assert not zk.any() and not zv.any()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D,rot", [(128, 128), (64, 64), (80, 32), (96, 20), (256, 128), (128, 6)])
def test_append_rotated(kind, inter, D, rot):
    rng = np.random.default_rng(D + rot)
    kvh, T = 2, 41
    wide = normal(rng, T, 5 * kvh * D)                # views of one projection output, as q | k | v leaves it
    cs = R.angles(rng.integers(0, 9000, T), R.np.power(10000.0, -np.arange(rot // 2) / (rot // 2)), 1.0).astype(np.float32)
    w = up(wide)
    kd = w[:, 3 * kvh * D:4 * kvh * D].unflatten(1, (kvh, D))
    vd = w[:, 4 * kvh * D:].unflatten(1, (kvh, D))
    c = make(kind, kvh, D, 2)
    slots = rng.permutation(128)[:T].astype(np.int32)
    q.kv_append(c, kd, vd, up(slots), cs=up(cs), interleaved=inter)
    gk, gv = q.kv_read(c, up(slots))
    k32 = R.rotate(kd.cpu().numpy(), cs, inter)        # the same separate fp32 roundings
    assert np.array_equal(gk.cpu().numpy(), R.stored(k32, kind))
    assert np.array_equal(gv.cpu().numpy(), R.stored(vd.cpu().numpy(), kind))


@pytest.mark.parametrize("kind", KINDS)
def test_append_stores_finite_values(kind):
    x = np.zeros((3, 1, 64), np.float32)
    x[0, 0, :6] = [np.nan, 1, np.inf, -np.inf, 1e30, 3]
    x[1, 0, :] = np.nan
    x[2, 0, 40] = 65520.0
    c = make(kind, 1, 64, 1)
    s = up(np.arange(3, dtype=np.int32))
    q.kv_append(c, up(x), up(x), s)
    for got in q.kv_read(c, s):
        assert np.array_equal(got.cpu().numpy(), R.stored(x, kind))
        assert torch.isfinite(got).all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [64, 80, 128, 256])
def test_move(kind, D):
    rng = np.random.default_rng(D)
    kvh, page, pages = 2, 64, 9
    c = make(kind, kvh, D, pages, page)
    n_all = pages * page
    k, v = (normal(rng, n_all, kvh, D) for _ in range(2))
    every = up(np.arange(n_all, dtype=np.int32))
    q.kv_append(c, up(k), up(v), every)
    rk, rv = (t.cpu().numpy() for t in q.kv_read(c, every))
    # group 0: an accepted path moved down over its own tree; 1: a cycle and a
    # shift; 2: padding and slots outside; 3: a slot onto itself
    src = -np.ones((4, 64), np.int32)
    dst = -np.ones((4, 64), np.int32)
    path = np.sort(rng.permutation(100)[:64])
    src[0], dst[0] = 60 + path, 60 + np.arange(64)
    src[1, :5], dst[1, :5] = [200, 201, 202, 210, 211], [201, 202, 200, 211, 212]
    src[2, :4], dst[2, :4] = [300, 9999, 301, -5], [310, 311, 99999, 312]
    src[3, 7], dst[3, 7] = 400, 400
    q.kv_move(c, up(src), up(dst))
    for got, r in zip(q.kv_read(c, every), (rk, rv)):
        want = r.copy()
        for s, d in zip(src.reshape(-1), dst.reshape(-1)):
            if 0 <= s < n_all and 0 <= d < n_all:
                want[d] = r[s]
        assert np.array_equal(got.cpu().numpy(), want)


def test_refusals_leave_everything():
    c = make("q8_0", 2, 64, 2)
    x = torch.ones(4, 2, 64, device=DEV)
    s = torch.arange(4, dtype=torch.int32, device=DEV)
    for bad in (lambda: q.kv_append(c, x, x.half(), s), lambda: q.kv_append(c, x[:, :1], x, s),
                lambda: q.kv_append(c, x, x, s.long()), lambda: q.kv_append(c, x, x, s[:3]),
                lambda: q.kv_append(c, x.transpose(0, 1), x, s), lambda: q.kv_append(c, x.bfloat16(), x.bfloat16(), s),
                lambda: q.kv_append(c, x, x, s, cs=torch.zeros(4, 33, 2, device=DEV)),
                lambda: q.kv_append(c, x, x, s, cs=torch.zeros(3, 32, 2, device=DEV)),
                lambda: q.kv_read(c, s, torch.bfloat16), lambda: q.kv_move(c, s[None], s[None, :3]),
                lambda: q.kv_move(c, torch.zeros(1, 65, dtype=torch.int32, device=DEV),
                                  torch.zeros(1, 65, dtype=torch.int32, device=DEV)),
                lambda: q.rope(x, torch.zeros(4, 33, 2, device=DEV)), lambda: q.rope(x[..., :60], torch.zeros(4, 8, 2, device=DEV)),
                lambda: q.rope(x, torch.zeros(4, 8, 2, device=DEV), out=torch.empty(4, 2, 64, dtype=torch.float16, device=DEV))):
        with pytest.raises((ValueError, q.QmmError)):
            bad()
    assert (c.k == 255).all() and (c.v == 255).all()
