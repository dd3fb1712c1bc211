"""fp64 CPU definition of the calls over caches in pages (test infrastructure).

Row j*page + r of a slot is row r of page table[j] of the pools
[n_pages, Hkv, page, D].  A slot that holds L rows before a decode step sees
rows 0 .. L in it.
"""
from __future__ import annotations

import numpy as np


def append(q_raw, k_raw, pos, q_norm, k_norm, eps, rot, theta):
    """Rows at positions pos: normalised per head (weights None: not) and turned; q_raw, k_raw [n, H, D]."""
    def one(x, w):
        x = np.asarray(x, np.float64)
        if w is not None:
            x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(w, np.float64)
        y = x.copy()
        for j in range(rot // 2):
            a = np.asarray(pos, np.float64)[:, None] * theta ** (-2.0 * j / rot)
            c, s = np.cos(a), np.sin(a)
            y[..., j] = x[..., j] * c - x[..., j + rot // 2] * s
            y[..., j + rot // 2] = x[..., j + rot // 2] * c + x[..., j] * s
        return y
    return one(q_raw, q_norm), one(k_raw, k_norm)


def attend(K, V, table, L, q, scale, gate=None, places=None):
    """One slot's decode rows: q [Hq, D] over the pages of the pools; places: per KV
    head the listed table columns (None: all up to the row's own).  Returns the
    output, the sum of weights times |values| and the largest sum of |products| of a score."""
    _, Hkv, page, D = K.shape
    Hq = q.shape[0]
    G = Hq // Hkv
    out, mag, prod = np.zeros((Hq, D)), np.zeros((Hq, D)), 0.0
    for h in range(Hq):
        g = h // G
        cols = range(L // page + 1) if places is None else places[g]
        ks, vs = [], []
        for j in cols:
            n = min(page, L + 1 - j * page)
            if n > 0:
                ks.append(K[table[j], g, :n])
                vs.append(V[table[j], g, :n])
        if not ks:
            continue  # sees nothing: zeros
        k, v = np.concatenate(ks).astype(np.float64), np.concatenate(vs).astype(np.float64)
        s = (k @ q[h]) * scale
        w = np.exp(s - s.max())
        w /= w.sum()
        out[h], mag[h] = w @ v, w @ np.abs(v)
        prod = max(prod, float((np.abs(k) @ np.abs(q[h])).max() * scale))
    if gate is not None:
        f = 1 / (1 + np.exp(-gate))
        out, mag = out * f, mag * f
    return out, mag, prod


def bounds(keys):
    """codes [2, D] and exponent of one page's keys [page, D]."""
    keys = np.asarray(keys, np.float64)
    if not np.isfinite(keys).all():
        return np.zeros((2, keys.shape[1]), np.int64), 128
    top, e = np.abs(keys).max(), -100
    while top > 127 * 2.0 ** e:
        e += 1
    return np.stack([np.floor(keys.min(0) / 2.0 ** e), np.ceil(keys.max(0) / 2.0 ** e)]).astype(np.int64), e


def query_codes(q):
    """Queries of one KV head [G, D] in whole steps of one power of two."""
    q = np.asarray(q, np.float64)
    if not np.isfinite(q).all() or not q.any():
        return np.zeros(q.shape)
    top, e = np.abs(q).max(), -200
    while top > 127 * 2.0 ** e:
        e += 1
    return np.rint(q / 2.0 ** e)


def scores(q, codes, exps):
    """q [G, D], codes [n, 2, D], exps [n]."""
    u = query_codes(q)[:, None]
    s = np.where(u > 0, u * codes[None, :, 1], u * codes[None, :, 0]).sum(-1).max(0)
    return np.where(np.asarray(exps) >= 128, np.inf, np.ldexp(s, np.minimum(exps, 127)))


def select(q, codes, exps, nb, first, last, n_sel):
    """The pages of nb that are looked at; codes, exps of pages first .. nb - last - 1."""
    if nb <= n_sel:
        return list(range(nb))
    s = scores(q, codes, exps)
    ranked = sorted(range(len(s)), key=lambda j: (-s[j], j))[:n_sel - first - last]
    return sorted(list(range(first)) + [first + j for j in ranked] + list(range(nb - last, nb)))
