"""Plain 64-bit references of the rotary / cache / attention operators, in
numpy: definitions only, nothing of the library's layout."""
import numpy as np

import oracle
import qmm_inputs as G

F16 = 16
TYPES = {"f16": F16, "q8_0": G.Q8_0, "q4_0": G.Q4_0}


def angles(pos, freqs, m):
    a = np.asarray(pos, np.float64)[:, None] * np.asarray(freqs, np.float64)[None, :]
    return np.stack([m * np.cos(a), m * np.sin(a)], -1)


def rotate(x, cs, interleaved):
    """x [T, H, D] in the precision of cs [T, pairs, 2]."""
    y = np.array(x, dtype=cs.dtype)
    p = np.arange(cs.shape[1])
    i0, i1 = (2 * p, 2 * p + 1) if interleaved else (p, p + len(p))
    a, b, c, s = y[..., i0], y[..., i1], cs[:, None, :, 0], cs[:, None, :, 1]
    y[..., i0], y[..., i1] = a * c - b * s, b * c + a * s
    return y


def stored(x, kind):
    """What a cache of a type holds of fp32 rows [T, H, D], as fp64: the oracle's
    encoder and decoder on rows filled up with zeros."""
    x = np.nan_to_num(np.clip(np.where(np.isnan(x), 0, x), -65504, 65504)).astype(np.float32)
    if kind == "f16":
        return x.astype(np.float16).astype(np.float64)
    T, H, D = x.shape
    w = np.zeros((T * H, -(-D // 32) * 32), np.float32)
    w[:, :D] = x.reshape(T * H, D)
    t = TYPES[kind]
    return oracle.dequant(t, oracle.quantize(t, w), *w.shape)[:, :D].reshape(T, H, D).astype(np.float64)


def attend(q, k, v, see, scale):
    """q [T, H, D], k and v [L, Hkv, D], see bool [T, L] -> fp64 [T, H, D]."""
    T, H, D = q.shape
    g = H // k.shape[1]
    out = np.zeros((T, H, D))
    for h in range(H):
        s = scale * (q[:, h].astype(np.float64) @ k[:, h // g].T)
        s = np.where(see, s, -np.inf)
        m = s.max(-1, keepdims=True, initial=-np.inf)
        p = np.where(see, np.exp(s - np.where(np.isfinite(m), m, 0)), 0)
        l = p.sum(-1, keepdims=True)
        out[:, h] = np.where(l > 0, p @ v[:, h // g] / np.where(l > 0, l, 1), 0)
    return out


def tree(rng, n, back=6):
    """Parents of a random tree of n drafted tokens and the ancestor matrix."""
    par = [-1] + [int(rng.integers(max(-1, i - back), i)) for i in range(1, n)]
    see = np.eye(n, dtype=bool)
    for i, p in enumerate(par):
        if p >= 0:
            see[i] |= see[p]
    return par, see


def words(see, n_words=None):
    """bool [T, n] -> int64 [T, words]."""
    T, n = see.shape
    n_words = n_words or max(1, -(-n // 64))
    out = np.zeros((T, n_words), np.uint64)
    for j in range(min(n, 64 * n_words)):
        out[:, j // 64] |= see[:, j].astype(np.uint64) << np.uint64(j % 64)
    return out.view(np.int64)
