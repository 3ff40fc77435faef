"""fp64 NumPy oracle of the paged cache: the 8-bit row format, appending, reading back and
the attention of the last tokens of every sequence. Plain loops over sequences and heads."""
from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0


def e4m3_round(y):
    """Nearest e4m3 value (ties to even) of |y| <= 448: spacing 2^(e-3) in [2^e, 2^(e+1)),
    2^-9 below 2^-6. NaN stays NaN."""
    y = np.asarray(y, np.float64)
    mag = np.maximum(np.abs(y), 2.0 ** -6)
    step = np.exp2(np.floor(np.log2(np.where(np.isfinite(mag), mag, 1.0))) - 3)
    return np.round(y / step) * step


def e4m3_value(code):
    """Value of an e4m3 byte: sign, four exponent bits (bias 7), three fraction bits."""
    code = np.asarray(code, np.int64)
    s, e, f = code >> 7, (code >> 3) & 15, code & 7
    mag = np.where(e == 0, f * 2.0 ** -9, (8 + f) * np.exp2(e - 10.0))
    mag = np.where((e == 15) & (f == 7), np.nan, mag)
    return np.where(s == 1, -mag, mag)


def row_scale(x):
    """Power of two of each row of x [..., d]: the smallest s with max|x| / s <= 448 over
    finite values, at least 2^-126; 1 where the row holds no finite value but zero."""
    a = np.abs(np.asarray(x, np.float64))
    top = np.where(np.isfinite(a), a, 0.0).max(-1)
    frac, e = np.frexp(top / E4M3_MAX)          # top / 448 = frac * 2^e, frac in [1/2, 1)
    e = np.where(frac == 0.5, e - 1, e)         # an exact power of two is its own scale
    return np.where(top > 0, np.exp2(np.maximum(e, -126).astype(np.float64)), 1.0)


def quantise(x):
    """(values code, scale) of rows x [..., d] in the 8-bit format."""
    x = np.asarray(x, np.float64)
    s = row_scale(x)
    return e4m3_round(np.where(np.isfinite(x), x, np.nan) / s[..., None]), s


def append(pages, scales, x, table, start, count, page):
    """x [B,H,T,d] into pages [P,H,page,d] (and scales [P,H,page], or None): in place."""
    for b in range(x.shape[0]):
        for t in range(count[b]):
            pos = start[b] + t
            pg, row = table[b][pos // page], pos % page
            if scales is None:
                pages[pg, :, row] = x[b, :, t]
            else:
                pages[pg, :, row], scales[pg, :, row] = quantise(x[b, :, t])


def rows(pages, scales, table_row, n, h, page):
    """The first n rows of a sequence, head h: [n, d]."""
    if n == 0:
        return np.zeros((0, pages.shape[-1]))
    pos = np.arange(n)
    pg = np.asarray(table_row)[pos // page]
    x = pages[pg, h, pos % page].astype(np.float64)
    return x if scales is None else x * scales[pg, h, pos % page][:, None]


def decode(q, kp, vp, ks, vs, table, lens, page, scale, kept=None):
    """(out [B,Hq,T,d], lse [B,Hq,T], and for error bounds per row the largest |v| attended
    and the largest sum |q_c k_c|). kept[b][h]: logical pages kept, or None."""
    B, Hq, T, d = q.shape
    H = kp.shape[1]
    G = Hq // H
    out, lse = np.zeros((B, Hq, T, d)), np.full((B, Hq, T), -np.inf)
    vmax, qk = np.zeros((B, Hq, T)), np.zeros((B, Hq, T))
    for b in range(B):
        n = int(lens[b])
        for h in range(H):
            k, v = (rows(p, s, table[b], n, h, page) for p, s in ((kp, ks), (vp, vs)))
            ok = np.ones(n, bool)
            if kept is not None:
                ok = np.isin(np.arange(n) // page, np.asarray(kept[b][h], np.int64))
            for t in range(T):
                sees = ok & (np.arange(n) < n - (T - 1 - t))
                if not sees.any():
                    continue
                for g in range(h * G, (h + 1) * G):
                    x = np.asarray(q[b, g, t], np.float64)
                    l = scale * (k[sees] @ x)
                    m = l.max()
                    p = np.exp(l - m)
                    out[b, g, t] = p @ v[sees] / p.sum()
                    lse[b, g, t] = m + np.log(p.sum())
                    vmax[b, g, t] = np.abs(v[sees]).max()
                    qk[b, g, t] = (np.abs(k[sees]) @ np.abs(x)).max()
    return out, lse, vmax, qk
