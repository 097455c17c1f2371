"""Products of Q8_0 activations (gemv_q8) against the decoded weights and
activations in 64 bits: |y - exact| <= 2e-5 sum |w x|, as of qmm_gemv."""
import numpy as np
import pytest

import oracle
import qmm_inputs as G

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import dequant_matmul_amd as q  # noqa: E402

DEV = "cuda:0"
TYPES = (G.Q4_0, G.Q8_0, G.Q4_K, G.Q6_K, G.Q5_0, G.Q5_K)
TOL = 2e-5


def up(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def activations(rng, batch, k):
    x = rng.standard_normal((batch, k)).astype(np.float32) * np.exp(rng.uniform(-6, 6, (batch, k // 32, 1))).repeat(32, 1).reshape(batch, k)
    return oracle.quantize(G.Q8_0, x.astype(np.float32))


def check(t, w, n, k, x, y):
    W, X = oracle.dequant(t, w, n, k).astype(np.float64), oracle.dequant(G.Q8_0, x, x.shape[0], k).astype(np.float64)
    ref, mag = X @ W.T, np.abs(X) @ np.abs(W).T
    y = y.cpu().numpy()
    assert y.shape == ref.shape and np.all(np.abs(y - ref) <= TOL * mag)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("n,blocks", [(1, 1), (3, 2), (5, 3), (17, 5), (64, 8), (100, 16), (513, 4), (31, 64), (9, 71),
                                      (40, 130), (6, 700)])
def test_against_64_bits(t, n, blocks):
    k = blocks * G.BLOCK_ELEMS[t] if blocks < 200 else min(blocks * G.BLOCK_ELEMS[t], 65536 + G.BLOCK_ELEMS[t])
    rng = np.random.default_rng(1000 * t + n + blocks)
    w = G.gen_weights(t, n, k, seed=n + blocks)
    for batch in ((1, 2, 3, 4, 5, 6, 7, 8) if blocks < 20 else (1, 3, 8)):
        x = activations(rng, batch, k)
        buf = torch.full((batch * n + 16,), 7.0, device=DEV)
        off = 4 if n % 4 else 8
        y = buf[off:off + batch * n].view(batch, n)
        q.gemv_q8(up(w), t, n, k, up(x), out=y)
        check(t, w, n, k, x, y)
        assert bool((buf[:off] == 7).all()) and bool((buf[off + batch * n:] == 7).all())


@pytest.mark.parametrize("t", TYPES)
def test_a_decoders_projections(t):
    rng = np.random.default_rng(t)
    for n, k in ((4096, 4096), (1024, 2048), (2048, 5632), (512, 14336)):
        w = G.gen_weights(t, n, k, seed=t + n)
        wd = up(w)
        for batch in (1, 5):
            x = activations(rng, batch, k)
            check(t, w, n, k, x, q.gemv_q8(wd, t, n, k, up(x)))


def test_a_row_does_not_depend_on_its_company():
    """Nor on the other problems, the batch or the call."""
    rng = np.random.default_rng(3)
    k, ns = 4096, [300, 7, 129, 64, 1000]
    types = [G.Q4_K, G.Q6_K, G.Q8_0, G.Q4_K, G.Q5_0]
    ws = [up(G.gen_weights(t, n, k, seed=n)) for t, n in zip(types, ns)]
    x = up(activations(rng, 8, k))
    outs = q.gemv_q8_multi(ws, types, ns, k, x)
    again = q.gemv_q8_multi(ws, types, ns, k, x)
    for w, t, n, o, p in zip(ws, types, ns, outs, again):
        assert torch.equal(o, p) and torch.equal(o, q.gemv_q8(w, t, n, k, x))
        for b in range(1, 9):
            assert torch.equal(o[:b], q.gemv_q8(w, t, n, k, x[:b].contiguous()))


def test_many_problems_of_a_type():
    rng = np.random.default_rng(4)
    k, ns = 512, [1, 2, 3, 0, 50, 6, 7, 8, 9, 10, 11, 12, 130, 14, 15, 16, 17, 64]
    host = [G.gen_weights(G.Q4_0, n, k, seed=n) if n else np.zeros((0, 1), np.uint8) for n in ns]
    x = activations(rng, 2, k)
    outs = q.gemv_q8_multi([up(h) for h in host], [G.Q4_0] * len(ns), ns, k, up(x))
    for h, n, o in zip(host, ns, outs):
        if n:
            check(G.Q4_0, h, n, k, x, o)
        assert o.shape == (2, n)


@pytest.mark.parametrize("t", TYPES)
def test_extreme_fields(t):
    """Every byte of the blocks drawn from its ends, scales of both signs, and
    activation codes of -128 and 127."""
    rng = np.random.default_rng(50 + t)
    n, k = 33, 4 * 256
    be, bb = G.BLOCK_ELEMS[t], G.BLOCK_BYTES[t]
    w = rng.choice(np.array([0, 255, 127, 128, 1], np.uint8), (n, k // be, bb))
    for at in ([208] if t == G.Q6_K else [0, 2] if t in (G.Q4_K, G.Q5_K) else [0]):
        d = rng.choice(np.array([1.0, -2.0, 0.0, 1e-3, 6e-8], np.float16), (n, k // be, 1))
        w[:, :, at:at + 2] = d.view(np.uint8)
    w = w.reshape(n, -1)
    x = rng.choice(np.array([0x80, 0x7f, 0, 1, 0xff], np.uint8), (4, k // 32, 34))
    x[:, :, :2] = rng.choice(np.array([1.0, -0.5, 0.0, 100.0, 6e-8], np.float16), (4, k // 32, 1)).view(np.uint8)
    x = x.reshape(4, -1)
    check(t, w, n, k, x, q.gemv_q8(up(w), t, n, k, up(x)))


@pytest.mark.parametrize("t", [G.Q4_K, G.Q5_K])
def test_rows_of_zero_weights_give_zero(t):
    """d sc q = dmin m for every element: nothing may be left of the difference."""
    rng = np.random.default_rng(7)
    n, k = 24, 8192
    w = np.zeros((n, k // 256, G.BLOCK_BYTES[t]), np.uint8)
    d = rng.uniform(1e-4, 1e-2, (n, k // 256, 1)).astype(np.float16)
    w[:, :, 0:2] = d.view(np.uint8)
    w[:, :, 2:4] = d.view(np.uint8)
    # sub-blocks 0..3: sc 13, m 13 * q with one q; 4..7 zero scale and min
    for r in range(n):
        code = r % 4 + 1
        w[r, :, 4:8], w[r, :, 8:12] = 13, 13 * code
        w[r, :, 16 if t == G.Q4_K else 48:] = code * 17
    w = w.reshape(n, -1)
    assert not oracle.dequant(t, w, n, k).any()
    y = q.gemv_q8(up(w), t, n, k, up(activations(rng, 3, k)))
    assert not y.any()


def test_cancelling_weights_keep_the_bar():
    """Weights that are small differences of large d sc q and dmin m."""
    rng = np.random.default_rng(9)
    n, k = 64, 4096
    w = G.gen_weights(G.Q4_K, n, k, seed=3).reshape(n, k // 256, 144)
    d = rng.uniform(1e-3, 1e-2, (n, k // 256, 1)).astype(np.float16)
    w[:, :, 0:2] = d.view(np.uint8)
    w[:, :, 2:4] = np.nextafter(d, np.float16(1)).view(np.uint8)
    w[:, :, 4:8], w[:, :, 8:12], w[:, :, 12:16] = 7, 63, 0x97        # 7 * 9 against 63; 7 * 9 against 9 (+ noise)
    w[:, :, 16:] = 0x99
    w = w.reshape(n, -1)
    x = activations(rng, 2, k)
    check(G.Q4_K, w, n, k, x, q.gemv_q8(up(w), G.Q4_K, n, k, up(x)))


def test_empty_sums():
    y = q.gemv_q8(torch.empty(0, dtype=torch.uint8, device=DEV), G.Q8_0, 5, 0, torch.empty(3, 0, dtype=torch.uint8, device=DEV))
    assert y.shape == (3, 5) and not y.any()
    assert q.gemv_q8(up(G.gen_weights(G.Q8_0, 5, 64, 1)), G.Q8_0, 5, 64, torch.empty(0, 68, dtype=torch.uint8, device=DEV)).shape == (0, 5)
    assert q.gemv_q8_multi([], [], [], 64, torch.empty(1, 68, dtype=torch.uint8, device=DEV)) == []


def test_weights_at_the_end_of_their_buffer():
    """Rows of 34 and 210 bytes whose last one ends where its storage does."""
    rng = np.random.default_rng(12)
    for t, n, k in ((G.Q8_0, 7, 32), (G.Q6_K, 3, 256), (G.Q5_0, 5, 96), (G.Q4_0, 9, 32), (G.Q6_K, 1, 4096 + 256)):
        w = G.gen_weights(t, n, k, seed=k)
        pad = -w.size % 16
        buf = up(np.concatenate([np.full(pad + 0, 255, np.uint8), w.reshape(-1)]))
        wd = buf[pad:] if buf[pad:].data_ptr() % 16 == 0 else up(w.reshape(-1))
        x = activations(rng, 2, k)
        check(t, w, n, k, x, q.gemv_q8(wd, t, n, k, up(x)))
