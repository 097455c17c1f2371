"""The operators of include/qst.h from their definitions, in integers and 64 bits
(numpy on the host)."""
import numpy as np

INT_MOST = 2 ** 31 - 1


def plan(table, ctx, fresh, free, count, tokens, page):
    """(table, qstart, slots, pos, granted, left), request after request."""
    table = table.copy()
    B, cols = table.shape
    pages = len(free)
    F = min(max(int(count), 0), pages)
    fresh = [1] * B if fresh is None else fresh
    slots, pos = np.full(tokens, -1, np.int32), np.zeros(tokens, np.int32)
    qstart, granted, asked, left, row = [0], [], 0, F, 0
    for b in range(B):
        c, t = int(ctx[b]), int(fresh[b])
        good = c >= 0 and t >= 0 and c + t <= min(cols * page, INT_MOST) and row + t <= tokens
        need = -(-(c + t) // page) - -(-c // page) if good else 0
        ok = good and (need == 0 or asked + need <= F)
        if ok:
            for i in range(need):
                table[b, -(-c // page) + i] = free[F - 1 - asked - i]
            left = F - asked - need if need else left
            p = np.arange(c, c + t)
            pg = table[b, p // page].astype(np.int64)
            slots[row:row + t] = np.where((pg >= 0) & (pg < pages), pg * page + p % page, -1)
            pos[row:row + t] = p
        granted.append(int(ok))
        asked += need
        row = min(row + max(t, 0), tokens + 1)
        qstart.append(min(row, tokens))
    return table, np.array(qstart, np.int32), slots, pos, np.array(granted, np.int32), left


def trim(table, held, kept, free, count, page):
    """(free, left)."""
    free = free.copy()
    F = min(max(int(count), 0), len(free))
    back = []
    for row, h, k in zip(table, held, kept):
        back += list(row[-(-max(int(k), 0) // page):min(-(-max(int(h), 0) // page), len(row))])
    if F + len(back) > len(free):
        return free, F
    free[F:F + len(back)] = back[::-1]
    return free, F + len(back)


def norm(x, res, w, eps):
    """(s, out) in 64 bits."""
    s = x.astype(np.float64) + (0 if res is None else res.astype(np.float64))
    y = s / np.sqrt((s * s).mean(-1, keepdims=True) + float(np.float32(eps)))
    return s, y * (1 if w is None else w.astype(np.float64))


def lora(x, adapter, qstart, targets, scale, ranks):
    """[(y, bound)] of (a, b, base) targets: bound is the sum of the products'
    magnitudes and the largest inner sum's (times |b|), both scaled."""
    x = x.astype(np.float64)
    out = []
    for a, b, base in targets:
        y, mag, top = base.astype(np.float64), np.zeros(base.shape), np.zeros(base.shape)
        for i, ad in enumerate(adapter):
            rows = slice(qstart[i], qstart[i + 1])
            if ad < 0 or ad >= len(a):
                continue
            r = a.shape[1] if ranks is None else max(0, min(int(ranks[ad]), a.shape[1]))
            s = 1.0 if scale is None else float(scale[ad])
            A, B = a[ad, :r].astype(np.float64), b[ad, :, :r].astype(np.float64)
            h = x[rows] @ A.T
            y[rows] += s * (h @ B.T)
            mag[rows] = abs(s) * (np.abs(x[rows]) @ np.abs(A).T) @ np.abs(B).T
            top[rows] = abs(s) * np.abs(h).max(-1, keepdims=True, initial=0) * np.abs(B).sum(-1)[None]
        out.append((y, mag, top))
    return out
