"""GPU tests of attention where the usual bars would hide a loss of accuracy:
score errors counted with the weight of their token, losses at the bottom of the
fp16 range with the largest product instead of the largest |v|.

p are the softmax weights of the reference, A = sum_j p_j |v_j|, e_j = sum_d |scale
q_d k_jd| the size of a score.  A score error of r e_j moves weight j by that factor,
and the sum of the weights with it, so the output by r S, S = sum_j p_j e_j (|v_j| + A).
  float32: q and the weights (times the V scale) in two fp16 parts, 2^-22 each, fp32
    sums of at most 2^8 products with half steps of 2^-24 a block and a tree over
    tiles and splits: 2^-19 S + 2^-18 A.
  float16, few rows: q exact; the weight (times the V scale) rounded once to fp16 and
    the output once, half a step of 2^-11 each: 2^-10 A on top.
  float16, many rows: K and V of a quantized cache rounded to fp16 too: 2^-11 S, and
    2^-11 A on top of that.
Below 2^-14 a half of a product has steps of 2^-24, an error of 2^-25 against a
reference of 2^10.  The reference lies at most 2^5 below the row's largest product p_j
s_j (s_j the largest V scale of token j, at least 2^-14), and at most 2^w above it, w
the spread of V scales up to which a tile is taken at one exponent (8 in float32, 16 in
float16), and another 2 for exponents rounded up: n 2^(w - 33) max_j p_j max(vmax_j,
2^-7) for n tokens, vmax_j the largest stored |v| of token j (a Q8_0 code reaches 127).
A float16 result below 2^-14 has an error of 2^-25.
"""
import numpy as np
import pytest

import kv_ref as R
import test_gpu_attention as A

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import dequant_matmul_amd as q  # noqa: E402

up, DEV = A.up, A.DEV


def put(c, b, k, v):
    """The K and V rows of sequence b written anew."""
    p = np.arange(len(k))
    slots = c.table[b, p // c.page] * c.page + p % c.page
    q.kv_append(c.cache, up(k.astype(np.float32)), up(v.astype(np.float32)), up(slots.astype(np.int32)))
    c.k[b], c.v[b] = R.stored(k, c.kind), R.stored(v, c.kind)


def judge(c, got, dt, b=0, rows=None, heads=None):
    """Rows (of sequence b) and heads of got within the bar; every bar must also
    refuse a result of zeros."""
    rows = np.arange(c.tq[b]) if rows is None else np.asarray(rows)
    at = c.starts[b] + rows
    heads = range(c.q.shape[1]) if heads is None else heads
    group = c.q.shape[1] // c.k[b].shape[1]
    few = max(c.tq) * group <= 32
    x = up(c.q[at]).to(dt).cpu().numpy().astype(np.float64)
    got = got[up(at)].cpu().numpy().astype(np.float64)
    worst, told = 0.0, False
    for h in heads:
        k, v = c.k[b][:, h // group], c.v[b][:, h // group]
        s = np.where(c.see[b][rows], x[:, h] @ k.T * c.D ** -0.5, -np.inf)
        m = s.max(-1, keepdims=True)
        p = np.exp(s - np.where(np.isfinite(m), m, 0))
        p /= np.maximum(p.sum(-1, keepdims=True), 1e-300)
        out, size = p @ v, p @ np.abs(v)
        pe = p * (np.abs(x[:, h]) @ np.abs(k).T * c.D ** -0.5)
        moved = pe @ np.abs(v) + size * pe.sum(-1, keepdims=True)
        w = 8 if dt == torch.float32 else 16
        low = len(k) * 2.0 ** (w - 33) * (p * np.maximum(np.abs(v).max(-1), 2.0 ** -7)).max(-1)[:, None]
        tol = 2.0 ** -19 * moved + 2.0 ** -18 * size + low
        if dt == torch.float16:
            tol += 2.0 ** -10 * size + 2.0 ** -25
            if not few and c.kind != "f16":
                tol += 2.0 ** -11 * (moved + size) + 2.0 ** -25
        off = np.abs(got[:, h] - out)
        assert not np.isnan(off).any()
        worst, told = max(worst, (off / tol).max()), told or (np.abs(out) > tol).any()
    assert worst <= 1, "%.3g of the bar" % worst
    assert told or not np.concatenate([c.see[b][rows]]).any()


@pytest.mark.parametrize("dt", A.DTS)
@pytest.mark.parametrize("kind", A.KINDS)
@pytest.mark.parametrize("tq", [1, 40])
@pytest.mark.parametrize("D", [64, 80, 128, 256])
def test_unlike_scales_of_v_in_one_tile(kind, dt, tq, D):
    """A token with values 2^27 times those of its 63 neighbours and no weight has no
    part in the result, and costs it no accuracy either."""
    c = A.Case(kind, [64], [tq], 2, 4, D, seed=50 + D)
    rng = np.random.default_rng(51)
    k, v = rng.standard_normal((2, 64 + tq, 2, D))
    k *= 0.05
    v *= 2.0 ** -12
    k[10], v[10] = 0, 60000.0
    k[10, :, :8] = -6.0 * D ** 0.5         # a score near -48 * 2
    c.q[..., :8] = 2.0
    put(c, 0, k, v)
    judge(c, c.run(dt), dt)


@pytest.mark.parametrize("dt", A.DTS)
@pytest.mark.parametrize("kind", A.KINDS)
@pytest.mark.parametrize("D", [8, 64, 80, 96, 128, 200, 256])
def test_single_tokens(kind, D, dt):
    c = A.Case(kind, [0, 1, 62, 63, 64, 127, 128, 300], [1] * 8, 2, 4, D, page=128, seed=D)
    got = c.run(dt)
    for b in range(8):
        judge(c, got, dt, b)


@pytest.mark.parametrize("dt", A.DTS)
@pytest.mark.parametrize("kind", A.KINDS)
@pytest.mark.parametrize("tq", [3, 8])
def test_few_rows_in_splits(kind, tq, dt):
    c = A.Case(kind, [2900, 40], [tq, tq], 2, 4, 128, page=64, seed=40 + tq, tree=True)
    got = c.run(dt)
    for b in range(2):
        judge(c, got, dt, b)


@pytest.mark.parametrize("dt", A.DTS)
@pytest.mark.parametrize("kind", A.KINDS)
@pytest.mark.parametrize("spread", [1e-6, 1.0, 30.0, 3000.0])
@pytest.mark.parametrize("tq", [5, 40])
def test_sharp_and_flat_softmax(kind, tq, spread, dt):
    if spread == 3000 and tq == 40 and dt == torch.float16 and kind != "f16":
        pytest.skip("K rounded to fp16 moves scores of 20000 by 10: no bar on the weights")
    c = A.Case(kind, [700], [tq], 2, 4, 128, seed=3, spread=spread, vscale=20.0)
    judge(c, c.run(dt), dt)


@pytest.mark.parametrize("dt,lift", [(torch.float32, n) for n in list(range(0, 27)) + [30, 60, 100]] +
                         [(torch.float16, n) for n in range(0, 25)])
@pytest.mark.parametrize("kind", A.KINDS)
@pytest.mark.parametrize("tq", [1, 40])
def test_scores_past_the_whole_numbers(kind, tq, dt, lift):
    """Scores of any finite size, whose steps in fp32 are wider than the softmax's unit: one
    token takes a row, or two of equal keys share it.  Keys are a_j in every dim, a_j whole;
    the next lower a_j is 2% lower, a score error 2^-19 of it."""
    D, n = 128, 200 + tq
    c = A.Case(kind, [200], [tq], 2, 4, D, seed=70)
    rng = np.random.default_rng(71)
    a = rng.integers(1, 62, n).astype(np.float64)
    a[[40, 130, 150]] = 64, 63, 64          # in the first and the third tile
    a[200:] = 1
    high = max(0, lift - 15) if dt == torch.float16 else 0       # q ends at 2^15: the rest is K's
    k = np.repeat(a[:, None, None], 2, 1) * np.ones(D) * 2.0 ** high
    v = rng.standard_normal((n, 2, D))
    c.q[:] = 2.0 ** (lift - high)
    c.q[::2, ::2] *= -1                      # there the lowest keys win
    put(c, 0, k, v)
    got = c.run(dt).cpu().numpy().astype(np.float64)
    for r in range(tq):
        for h in range(c.q.shape[1]):
            s = c.k[0][:201 + r, h // 4, 0] * np.sign(c.q[r, h, 0])
            hit = np.flatnonzero(s > s.max() - 0.2 * 2.0 ** high)
            if lift == 0 and s.max() < 0:
                continue                     # scores a few units apart: the usual bars' case
            x = c.v[0][hit, h // 4]
            tol = (2.0 ** -9 if dt == torch.float16 else 2.0 ** -18) * np.abs(x).mean(0) + (1e-4 if lift == 0 else 2.0 ** -24)
            assert np.all(np.abs(got[r, h] - x.mean(0)) <= tol), (r, h, len(hit))


@pytest.mark.parametrize("kind", A.KINDS)
@pytest.mark.parametrize("tq", [1, 8, 40])
@pytest.mark.parametrize("ctx", [200, 3000])
def test_values_at_the_end_of_fp16(kind, tq, ctx):
    """Every V at the largest stored value: a mean of them is that value, and no rounding of a
    weight takes an fp16 result past the range."""
    c = A.Case(kind, [ctx], [tq], 2, 4, 64, seed=90)
    v = np.full((ctx + tq, 2, 64), 65504.0)
    v[..., 1::2] *= -1
    k = c.k[0].copy()
    put(c, 0, k, v)
    got = c.run(torch.float16).cpu().numpy().astype(np.float64)
    assert np.isfinite(got).all()
    # K rounded once more than in c.k has no part in it; weights and V by half a step each
    want = np.minimum(np.abs(c.v[0][0, 0]), 65504.0)
    assert np.all(np.abs(np.abs(got) - want) <= 2.0 ** -10 * want + 32)
    assert np.all(np.sign(got) == np.sign(v[0, 0]))


@pytest.mark.parametrize("kind", ["f16", "q8_0"])
@pytest.mark.parametrize("tq", [1, 40])
def test_queries_at_the_end_of_fp32(kind, tq):
    """Queries whose scaled values lie just below the largest fp32, against keys so small
    that scores stay below it: the largest key takes the row."""
    D, n = 128, 100 + tq
    c = A.Case(kind, [100], [tq], 1, 4, D, seed=95)
    a = 1.0 + np.arange(n) % 32
    a[70] = 64
    k = np.zeros((n, 1, D))
    k[:, 0, :4] = a[:, None] * 2.0 ** -8        # (in four dims: the sum is 2^-8 of a value)
    v = np.random.default_rng(96).standard_normal((n, 1, D))
    put(c, 0, k, v)
    c.q[:] = 2.2e38
    got = c.run(torch.float32, scale=1.0).cpu().numpy()
    assert np.all(np.abs(got - c.v[0][70, 0]) <= 2.0 ** -18 * np.abs(c.v[0][70, 0]) + 2.0 ** -24)
