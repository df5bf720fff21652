"""The stand-alone operators from their definitions, in numpy at 64 bits."""
import numpy as np

E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6])
BLOCK = {"mxfp4": 32, "nvfp4": 16}


def nearest_even(a, table):
    """Index of the value of `table` (ascending) nearest to each a >= 0, ties to the even index, saturating."""
    mid = (table[1:] + table[:-1]) / 2
    up = np.searchsorted(mid, a, side="left")            # borders below a
    tie = (up < len(mid)) & (mid[np.minimum(up, len(mid) - 1)] == a)
    return np.where(tie & (up % 2 == 1), up + 1, up)


def e4m3_table():
    c = np.arange(127)
    e, f = c >> 3, c & 7
    return np.where(e > 0, (1 + f / 8) * 2.0 ** (e - 7.0), f * 2.0 ** -9)


def quantize(x, fmt, per=1):
    """(codes [n, K] one to an element, scale codes, G or None, values) of x float64 [n, K]."""
    n, K = x.shape
    v = x.reshape(n, -1, BLOCK[fmt])
    bad = ~np.isfinite(v).all(2)
    fin = np.where(np.isfinite(v), v, 0.0)
    amax = np.where(bad, 0.0, np.abs(fin).max(2))
    G = None
    if fmt == "mxfp4":
        with np.errstate(divide="ignore"):
            X = np.where(amax > 0, np.frexp(amax)[1] - 3, -126)
        X = np.clip(X, -126, 127)
        sc = np.where(bad, 255, X + 127)
        d = 2.0 ** X
    else:
        top = amax.reshape(n // per, -1).max(1)
        m, e = np.frexp(top / 2688)
        e = np.maximum(np.where(m == 0.5, e - 1, e), -100)
        G = np.where(top > 0, 2.0 ** e, 1.0)
        g = np.repeat(G, per)[:, None]
        tab = e4m3_table()
        idx = nearest_even(amax / (6 * g), tab)
        sc = np.where(bad, 127, idx)
        d = tab[idx] * g
    q = np.where(d[..., None] > 0, np.abs(fin) / np.where(d > 0, d, 1)[..., None], 0)
    idx = nearest_even(q, E2M1)
    idx = np.where(bad[..., None], 0, idx)
    neg = np.signbit(fin) & ~bad[..., None] & (d[..., None] > 0)
    val = np.where(neg, -1, 1) * E2M1[idx] * d[..., None]
    val = np.where(bad[..., None], np.nan, val)
    return (idx + 8 * neg).reshape(n, K).astype(np.uint8), sc.astype(np.uint8), G, val.reshape(n, K)


def pack(c):
    return (c[:, 0::2] | (c[:, 1::2] << 4)).astype(np.uint8)


def values(codes, scales, G, fmt, per=1):
    """float64 [n, K] of packed codes [n, K/2] and scale codes."""
    n = codes.shape[0]
    nib = np.stack([codes & 15, codes >> 4], 2).reshape(n, -1)
    v = np.where(nib & 8, -1.0, 1.0) * E2M1[nib & 7]
    if fmt == "mxfp4":
        d = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    else:
        tab = np.concatenate([e4m3_table(), [np.nan]])
        d = np.where(scales & 128, -1.0, 1.0) * tab[scales & 127] * np.repeat(G.astype(np.float64), per)[:, None]
    return v * np.repeat(d, BLOCK[fmt], axis=1)


def sort_pairs(ids, E):
    f = ids.reshape(-1).astype(np.int64)
    kept = (f >= 0) & (f < E)
    order = np.argsort(np.where(kept, f, E), kind="stable")
    n = int(kept.sum())
    counts = np.bincount(f[kept], minlength=E)
    perm = np.full(f.size, -1)
    perm[:n] = order[:n]
    inv = np.full(f.size, -1)
    inv[order[:n]] = np.arange(n)
    return counts, np.concatenate([[0], np.cumsum(counts)]), perm, inv.reshape(ids.shape)


def dispatch(x, inv, xs):
    out = xs.copy()
    t, j = np.nonzero((inv >= 0) & (inv < xs.shape[0]))
    out[inv[t, j]] = x[t]
    return out


def combine(ys, inv, gates):
    """(y, sum of the terms' magnitudes)."""
    T, k = inv.shape
    y, s = np.zeros((T, ys.shape[1])), np.zeros((T, ys.shape[1]))
    for j in range(k):
        t = np.nonzero((inv[:, j] >= 0) & (inv[:, j] < ys.shape[0]))[0]
        term = gates[t, j][:, None] * ys[inv[t, j]]
        y[t] += term
        s[t] += np.abs(term)
    return y, s


def combine_backward(dy, ys, inv, gates, dys):
    """(dys, dgates, sum of the magnitudes of dgates's terms)."""
    out, dg, s = dys.copy(), np.zeros(inv.shape), np.zeros(inv.shape)
    for j in range(inv.shape[1]):
        t = np.nonzero((inv[:, j] >= 0) & (inv[:, j] < ys.shape[0]))[0]
        r = inv[t, j]
        out[r] = gates[t, j][:, None] * dy[t]
        dg[t, j] = (dy[t] * ys[r]).sum(1)
        s[t, j] = np.abs(dy[t] * ys[r]).sum(1)
    return out, dg, s


def matmul(x, w, offsets, y):
    """(y, sum of the terms' magnitudes): x [n, K], w [g, N, K] float64."""
    out, s = y.copy(), np.zeros_like(y)
    for g in range(w.shape[0]):
        a, b = int(offsets[g]), int(offsets[g + 1])
        out[a:b] = x[a:b] @ w[g].T
        s[a:b] = np.abs(x[a:b]) @ np.abs(w[g]).T
    return out, s
