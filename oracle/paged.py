"""fp64 definition of the paged-cache operators: E4M3 rows with power-of-two scales, append,
read, keep, and the attention of new tokens over the cache.  numpy on the CPU, plain loops; shares
no code with the kernels."""

from __future__ import annotations

import numpy as np

# the finite E4M3 magnitudes by code 0 .. 126 (code 127 is NaN)
_MAG = np.array([(m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                 for e in range(16) for m in range(8)][:127])


def e4m3_values(codes: np.ndarray) -> np.ndarray:
    c = codes.astype(np.int64)
    mag = np.concatenate([_MAG, [np.nan]])[c & 127]
    return np.where(c & 128, -mag, mag)


def quantise_row(x: np.ndarray, top: float):
    """(codes uint8, scale code) of one row; ``top``: the largest magnitude that is stored."""
    x = np.asarray(x, dtype=np.float64)
    finite = np.isfinite(x)
    y = np.where(finite, np.clip(x, -top, top), 0.0)
    amax = float(np.abs(y).max()) if y.size else 0.0
    e = -126
    while amax > 448.0 * 2.0 ** e:
        e += 1
    y = y / 2.0 ** e
    codes = np.empty(x.shape, dtype=np.uint8)
    for i, (v, ok) in enumerate(zip(y, finite)):
        if not ok:
            codes[i] = 127
            continue
        d = np.abs(_MAG - abs(v))
        best = np.flatnonzero(d == d.min())
        c = int(best[0]) if len(best) == 1 else int(next(b for b in best if b % 2 == 0))   # ties to even
        codes[i] = c | (128 if np.signbit(x[i]) else 0)
    return codes, e + 127


def slot(table, b, pos, page):
    return int(table[b, pos // page]), pos % page


def gather(x, table, b, n, page):
    """Positions 0 .. n - 1 of sequence b of a [pages, Hk, page, ...] array: [Hk, n, ...]."""
    out = np.empty((x.shape[1], n) + x.shape[3:], dtype=x.dtype)
    for p in range(n):
        i, r = slot(table, b, p, page)
        out[:, p] = x[i, :, r]
    return out


def visible(n: int, bits=None) -> np.ndarray:
    """[n, n] visibility among new tokens: a chain, or bit j of the words of row t."""
    if bits is None:
        return np.tril(np.ones((n, n), dtype=bool))
    v = np.zeros((n, n), dtype=bool)
    for t in range(n):
        for j in range(n):
            v[t, j] = (int(bits[t, j // 64]) >> (j % 64)) & 1
    return v


def attend(q, k, v, length, scale, bits=None):
    """One sequence: q [T, Hq, d], k, v [Hk, length + T, d] (fp64), visibility bits [T, words] or
    None.  Returns O [T, Hq, d], LSE [T, Hq], and for error bounds A = sum_j p_j |v_j| (like O),
    W = sum of |v_j| over visible keys (like O) and R = max_j scale * sum_c |q_c k_jc| (like LSE)."""
    T, Hq, d = q.shape
    G = Hq // k.shape[0]
    see = np.concatenate([np.ones((T, length), dtype=bool), visible(T, bits)], axis=1)
    o, a, w = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape)
    lse, r = np.full((T, Hq), -np.inf), np.zeros((T, Hq))
    with np.errstate(invalid="ignore"):
        for t in range(T):
            idx = np.flatnonzero(see[t])
            if len(idx) == 0:
                continue
            for h in range(Hq):
                kk, vv = k[h // G, idx], v[h // G, idx]
                s = scale * (kk @ q[t, h])
                m = s.max()
                p = np.exp(s - m)
                z = p.sum()
                lse[t, h] = m + np.log(z)
                o[t, h] = (p / z) @ vv
                a[t, h] = (p / z) @ np.abs(vv)
                w[t, h] = np.abs(vv).sum(0)
                r[t, h] = (scale * (np.abs(kk) @ np.abs(q[t, h]))).max()
    return o, lse, a, w, r
