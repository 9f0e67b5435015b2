"""Oracle of the operators for drafts and bounded pages: attention of a tree of
drafted tokens, the packing of the accepted ones, the attention weight that each
cached row has drawn, and the eviction by it.  Plain numpy in 64 bits, one
branch and one head at a time; shares no code with the CUDA library.
"""
from __future__ import annotations

import numpy as np

from .branch_oracle import seen


def above(parent, i):
    """Draft i and those it hangs on."""
    path = []
    while i >= 0:
        path.append(i)
        i = int(parent[i])
    return path[::-1]


def _row(table, b, p, page):
    return int(table[b, p // page]), p % page


def _rows(x, table, b, h, n):
    """The first n rows of branch b and head h."""
    page = x.shape[2]
    return np.array([x[table[b, p // page], h, p % page] for p in range(n)], np.float64).reshape((n,) + x.shape[3:])


def tree_attention(q, cu, parent, prefix, K, V, table, length, scale):
    """out [Hq][N][D], lse [Hq][N] (rows of padding tokens: nan), and for error
    bounds the sum of p |v| per output, the largest scale sum |q k| of a row, and
    the keys of a row."""
    Hq, N, D = q.shape
    H = K.shape[1]
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
            kb, vb = _rows(K, table, b, h, full), _rows(V, table, b, h, full)
            for i in range(n):
                at = [p for p in range(full - n)] + [full - n + j for j in above(parent[lo:lo + n], i)]
                at = [p for p in at if p >= 0]
                k, v = np.concatenate((pk, kb[at])), np.concatenate((pv, vb[at]))
                bb = np.concatenate((bias, np.zeros(len(at))))
                ok = bb > -np.inf
                k, v, bb = k[ok], v[ok], bb[ok]
                for e in range(h * g, (h + 1) * g):
                    x = scale * (k @ q[e, lo + i]) + bb
                    if not len(x):
                        out[e, lo + i], lse[e, lo + i] = 0.0, -np.inf
                        continue
                    top = x.max()
                    w = np.exp(x - top)
                    lse[e, lo + i] = top + np.log(w.sum())
                    w /= w.sum()
                    out[e, lo + i] = w @ v
                    mag[e, lo + i] = w @ np.abs(v)
                    big[e, lo + i] = scale * (np.abs(k) @ np.abs(q[e, lo + i])).max()
                    keys[e, lo + i] = len(x)
    return out, lse, mag, big, keys


def page_keep(K, V, cu, rows, cu_keep, table, length):
    """Pages (changed in place) with the kept tokens' rows moved to the front of
    the new positions."""
    page = K.shape[2]
    for b in range(len(length)):
        past = int(length[b]) - int(cu[b + 1] - cu[b])
        for j, r in enumerate(rows[cu_keep[b]:cu_keep[b + 1]]):
            src, dst = _row(table, b, past + int(r) - int(cu[b]), page), _row(table, b, past + j, page)
            for x in (K, V):
                x[dst[0], :, dst[1]] = x[src[0], :, src[1]]


def page_mass(K, q, lse, rows, cu, table, length, scale, block, decay, mass, born=None, total=None):
    """mass (64 bits, changed in place) and born with the weights of the tokens,
    and the bound of each mass's relative error per unit of 2^-23 (see the
    tests): [n_pages][H][page], sum of w (D + 4) X + 2 (|lse| + X) + 4 + rows."""
    Hq, N, D = q.shape
    H, page = K.shape[1], K.shape[2]
    g = Hq // H
    q, lse = np.asarray(q, np.float64), np.asarray(lse, np.float64)
    err = np.zeros_like(mass)
    for b in range(len(length)):
        lo, n, full = int(cu[b]), int(cu[b + 1] - cu[b]), int(length[b])
        if n == 0:
            continue
        at = np.arange(lo, lo + n) if rows is None else np.asarray(rows[lo:lo + n], np.int64)
        sees = np.array([seen(i, n, full, block) for i in range(n)])
        p = np.arange(full)
        where = np.asarray(table[b], np.int64)[p // page], p % page
        for h in range(H):
            k = _rows(K, table, b, h, full)
            drew, off = np.zeros(full), np.zeros(full)
            for e in range(h * g, (h + 1) * g):
                s = lse[e, at][:, None]
                hidden = (p[None] >= sees[:, None]) | (s == -np.inf)
                with np.errstate(over="ignore", invalid="ignore"):
                    w = np.where(hidden, 0.0, np.exp(scale * (q[e, at] @ k.T) - s))
                    X = scale * (np.abs(q[e, at]) @ np.abs(k).T)
                    drew += w.sum(0)
                    off += np.where(hidden, 0.0, w * ((D + 4) * X + 2 * (np.abs(s) + X) + 4 + n * g)).sum(0)
            fresh = p >= full - n
            mass[where[0], h, where[1]] = np.where(fresh, 0.0, decay * mass[where[0], h, where[1]]) + drew
            err[where[0], h, where[1]] = off + 2 * mass[where[0], h, where[1]]
            if born is not None:
                a, c = where[0][fresh], where[1][fresh]
                born[a, h, c] = int(total[b]) - full + p[fresh]
    return err * 2.0 ** -23


def page_evict(arrays, mass, born, total, table, length, budget, first, recent):
    """arrays ([n_pages][H][page]..., changed in place): the rows that leave are
    overwritten by the kept ones from the budget on."""
    page, H = mass.shape[2], mass.shape[1]
    for b in range(len(length)):
        n = int(length[b])
        if n <= budget:
            continue
        for h in range(H):
            at = [_row(table, b, p, page) for p in range(n)]
            order = []
            for p, (i, r) in enumerate(at):
                age, last = (p, n) if born is None else (int(born[i, h, r]), int(total[b]))
                safe = age < first or age >= last - recent
                x = float(mass[i, h, r])
                order.append((not safe, 0.0 if safe else (-x if x == x else np.inf), 0 if x == x else 1, p))
            kept = {t[3] for t in sorted(order)[:budget]}
            holes = [p for p in range(budget) if p not in kept]
            for dst, src in zip(holes, sorted(p for p in kept if p >= budget)):
                for x in arrays:
                    x[at[dst][0], h, at[dst][1]] = x[at[src][0], h, at[src][1]]
