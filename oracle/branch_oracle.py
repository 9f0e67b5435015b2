"""Oracle of the branched-rollout operators: rotary positions with several
axes, the append to pages, and the attention of branches over a shared
prefix.  Plain numpy in 64 bits, one branch and one head at a time; shares no
code with the CUDA library.
"""
from __future__ import annotations

import numpy as np


def ladder(dims, base=10000.0):
    """Radians per position of each pair, axis after axis."""
    return np.concatenate([base ** (-2.0 * np.arange(d // 2) / max(d, 1)) for d in dims])


def rope(x, pos, dims, freqs, halves, inverse=False):
    """Rows x [H][N][D] turned by pos [N][axes]."""
    y = np.array(x, dtype=np.float64)
    axis = np.repeat(np.arange(len(dims)), [d // 2 for d in dims])
    n = len(axis)
    angle = np.asarray(pos, np.float64)[:, axis] * np.asarray(freqs)
    c, s = np.cos(angle), np.sin(angle) * (-1.0 if inverse else 1.0)
    i = np.arange(n)
    a, b = (i, i + n) if halves else (2 * i, 2 * i + 1)
    x0, x1 = np.array(y[..., a]), np.array(y[..., b])
    y[..., a], y[..., b] = x0 * c - x1 * s, x0 * s + x1 * c
    return y


def page_append(K, V, k, v, cu, table, length):
    """Pages K, V [n_pages][H][page][D] (changed in place) with the new rows
    k, v [H][N][D], already turned."""
    page = K.shape[2]
    for b in range(len(length)):
        n = int(cu[b + 1] - cu[b])
        for i in range(n):
            p = int(length[b]) - n + i
            at = int(table[b, p // page])
            K[at, :, p % page] = k[:, cu[b] + i]
            V[at, :, p % page] = v[:, cu[b] + i]


def seen(i, n, length, block):
    """Positions of its branch that new token i of n sees."""
    if not block:
        return length
    t = length - n + i
    return 0 if t < 0 else min(length, (t // block + 1) * block)


def branch_attention(q, cu, prefix, K, V, table, length, scale, block=0, bounds=False):
    """out [Hq][N][D] and lse [Hq][N] (rows of padding tokens: nan).

    prefix: None or (pK, pV [H][C][D], m [H][C] or None, size [H] or None).
    bounds: also the sum of p |v| per output, the largest scale sum |q k| of a
    row, and the keys of a row, for error bounds."""
    Hq, N, D = q.shape
    H, page = K.shape[1], K.shape[2]
    g = Hq // H
    q = np.asarray(q, np.float64)
    out, lse = np.full((Hq, N, D), np.nan), np.full((Hq, N), np.nan)
    mag, big, keys = np.zeros((Hq, N, D)), np.zeros((Hq, N)), np.zeros((Hq, N))
    for h in range(H):
        pk = pv = np.zeros((0, D))
        bias = np.zeros(0)
        if prefix is not None:
            pK, pV, m, size = prefix
            live = pK.shape[1] if size is None else int(size[h])
            pk, pv = np.asarray(pK[h, :live], np.float64), np.asarray(pV[h, :live], np.float64)
            with np.errstate(divide="ignore"):
                bias = np.zeros(live) if m is None else np.log(np.maximum(np.asarray(m[h, :live], np.float64), 0))
        for b in range(len(length)):
            lo, n, full = int(cu[b]), int(cu[b + 1] - cu[b]), int(length[b])
            if n == 0:
                continue
            most = seen(n - 1, n, full, block)
            p = np.arange(most)
            at = np.asarray(table[b], np.int64)[p // page] if most else np.zeros(0, np.int64)
            kk = np.concatenate((pk, np.asarray(K[at, h, p % page], np.float64).reshape(-1, D)))
            vv = np.concatenate((pv, np.asarray(V[at, h, p % page], np.float64).reshape(-1, D)))
            for e in range(h * g, (h + 1) * g):
                x = scale * (q[e, lo:lo + n] @ kk.T)
                x[:, :len(bias)] += bias
                sees = np.array([seen(i, n, full, block) for i in range(n)])
                x[:, len(bias):][p[None] >= sees[:, None]] = -np.inf
                with np.errstate(invalid="ignore", divide="ignore"):
                    top = x.max(1, initial=-np.inf, keepdims=True)
                    w = np.where(x == -np.inf, 0.0, np.exp(x - np.where(np.isfinite(top), top, 0)))
                    s = w.sum(1, keepdims=True)
                    w = np.where(s > 0, w / s, 0.0)
                    lse[e, lo:lo + n] = np.where(s > 0, top + np.log(s), -np.inf)[:, 0]
                out[e, lo:lo + n] = w @ vv
                if bounds:
                    mag[e, lo:lo + n] = w @ np.abs(vv)
                    big[e, lo:lo + n] = (scale * (np.abs(q[e, lo:lo + n]) @ np.abs(kk.T))).max(1, initial=0)
                    keys[e, lo:lo + n] = len(bias) + sees
    return (out, lse, mag, big, keys) if bounds else (out, lse)
