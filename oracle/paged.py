"""fp64 definitions of the paged-cache operators (dllm_paged_append, dllm_paged_attention) and
of the token sampling (dllm_sample), one row at a time in numpy.

Arrays are plain numpy; dtypes narrower than fp64 are widened on entry and nothing is rounded,
so a test adds the roundings of the side it checks to its tolerance.
"""
from __future__ import annotations

import numpy as np


def rows_of(q_start, kv_len, T):
    """(sequence, position) of each of T rows; (-1, -1) for rows of no sequence."""
    out = np.full((T, 2), -1, np.int64)
    for b in range(len(kv_len)):
        for t in range(max(0, int(q_start[b])), min(T, int(q_start[b + 1]))):
            out[t] = b, int(kv_len[b]) - (int(q_start[b + 1]) - t)
    return out


def normed(x, gamma, eps):
    x = np.asarray(x, np.float64)
    if gamma is None:
        return x
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(gamma, np.float64)


def rotated(x, pos, inv_freq):
    """x [heads, hd] turned by pos * inv_freq (rotate-half pairs)."""
    if inv_freq is None:
        return x
    h = x.shape[-1] // 2
    a = float(pos) * np.asarray(inv_freq, np.float64)
    c, s = np.cos(a), np.sin(a)
    return np.concatenate([x[:, :h] * c - x[:, h:] * s, x[:, h:] * c + x[:, :h] * s], -1)


def append(K, V, K_pages, V_pages, table, q_start, kv_len, Q=None, Q_out=None, gamma_q=None, gamma_k=None,
           eps=1e-5, inv_freq=None):
    """-> (K_pages, V_pages, Q_out or None, number of rows without a page); inputs untouched."""
    Kp, Vp = np.array(K_pages, np.float64), np.array(V_pages, np.float64)
    Qo = None if Q is None else np.array(Q_out, np.float64)
    page, lost = Kp.shape[1], 0
    for t, (b, pos) in enumerate(rows_of(q_start, kv_len, len(K))):
        if b < 0 or pos < 0:
            continue
        if Q is not None:
            Qo[t] = rotated(normed(Q[t], gamma_q, eps), pos, inv_freq)
        pg = int(table[b, pos // page]) if pos // page < table.shape[1] else -1
        if not 0 <= pg < len(Kp):
            lost += 1
            continue
        Kp[pg, pos % page] = rotated(normed(K[t], gamma_k, eps), pos, inv_freq)
        Vp[pg, pos % page] = np.asarray(V[t], np.float64)
    return Kp, Vp, Qo, lost


def attention(Q, K_pages, V_pages, table, q_start, kv_len, mask_block=0, scale=None):
    """-> (A, A_abs = the same weights over |V|, lse, n = keys seen), [T, n_q, hd] / [T, n_q] /
    [T]; rows of no sequence stay NaN."""
    Q = np.asarray(Q, np.float64)
    T, n_q, hd = Q.shape
    n_pages, page, n_kv, _ = K_pages.shape
    scale = 1.0 / np.sqrt(hd) if scale is None else scale
    A, Aa = np.full(Q.shape, np.nan), np.full(Q.shape, np.nan)
    lse, n = np.full((T, n_q), np.nan), np.zeros(T, np.int64)
    for t, (b, pos) in enumerate(rows_of(q_start, kv_len, T)):
        if b < 0:
            continue
        end = min(max(0, int(kv_len[b])), table.shape[1] * page)
        if mask_block > 0:
            end = min(end, (pos // mask_block + 1) * mask_block) if pos >= 0 else 0
        j = np.arange(end)
        pg = np.asarray(table[b])[j // page].astype(np.int64)
        j, pg = j[(pg >= 0) & (pg < n_pages)], pg[(pg >= 0) & (pg < n_pages)]
        n[t] = len(j)
        if len(j) == 0:
            A[t], Aa[t], lse[t] = 0.0, 0.0, -np.inf
            continue
        k = np.asarray(K_pages[pg, j % page], np.float64)
        v = np.asarray(V_pages[pg, j % page], np.float64)
        for h in range(n_q):
            g = h // (n_q // n_kv)
            s = k[:, g] @ Q[t, h] * scale
            w = np.exp(s - s.max())
            lse[t, h] = s.max() + np.log(w.sum())
            w /= w.sum()
            A[t, h] = w @ v[:, g]
            Aa[t, h] = w @ np.abs(v[:, g])
    return A, Aa, lse, n


def sample_row(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """-> (token, prob) of one row of logits; the scaled logits are rounded to fp32 by definition."""
    l = np.asarray(logits, np.float32)
    ok = ~np.isnan(l) & (l != -np.inf)
    if not ok.any():
        return -1, 0.0
    with np.errstate(divide="ignore", over="ignore"):
        inv = np.float32(1.0) / np.float32(temperature)
    if not (temperature > 0 and inv < np.inf):   # NaN, <= 0, or 1 / T past the fp32 range
        return int(np.flatnonzero(ok & (l == l[ok].max()))[0]), 1.0
    with np.errstate(invalid="ignore", over="ignore"):
        z = np.where(ok, l * inv, np.float32(-np.inf)).astype(np.float64)
        top = z.max()
        w = np.where(z == top, 1.0, np.exp(np.minimum(z - top, 0.0))) if np.isfinite(top) else (z == top) * 1.0
    order = np.lexsort((np.arange(len(z)), -z))
    order = order[z[order] > -np.inf]
    ws = w[order]
    if 0 < top_k < len(z):
        order, ws = order[:top_k], ws[:top_k]
    keep = np.ones(len(order), bool)
    if top_p < 1:
        c = np.cumsum(ws)
        keep &= (c - ws) < float(np.float32(top_p)) * c[-1]
    if min_p > 0:
        keep &= ws >= min(float(np.float32(min_p)), 1.0)
    keep[0] = True
    ids = np.sort(order[keep])
    c = np.cumsum(w[ids])
    uu = float(u) if u > 0 else 0.0
    i = min(int(np.searchsorted(c, uu * c[-1], side="right")), len(ids) - 1)
    while w[ids[i]] == 0:
        i -= 1
    return int(ids[i]), float(w[ids[i]] / c[-1])
