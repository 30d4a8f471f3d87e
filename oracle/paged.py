"""fp64 definitions of the paged-cache operators (dllm_paged_append, dllm_paged_attention, their forms over
8-bit pages) and of the token sampling (dllm_sample), one row at a time in numpy.

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


# ---------------------------------------------------------------------------- 8-bit pages
def e4m3(x):
    """x rounded to the nearest E4M3 value (ties to even, saturated at 448; NaN stays)."""
    x = np.asarray(x, np.float64)
    m = np.minimum(np.abs(x), 448.0)
    step = np.exp2(np.maximum(np.floor(np.log2(np.where(m > 0, m, 1.0))), -6) - 3)
    with np.errstate(invalid="ignore"):
        return np.copysign(np.minimum(np.rint(m / step) * step, 448.0), x)


def exponent_for(top):
    """The least exponent from -64 to 63 with top <= 448 * 2^e."""
    e = -64
    while e < 63 and top > 448.0 * 2.0 ** e:
        e += 1
    return e


def append_f8(K, V, K_codes, V_codes, K_exp, V_exp, table, q_start, kv_len, Q=None, Q_out=None, gamma_q=None, gamma_k=None,
              eps=1e-5, inv_freq=None, pos_base=None):
    """Codes [n_pages, page, n_kv, hd] as values, exponents [n_pages, n_kv] -> (dict of K and V: codes before
    their last rounding, exponents, and whether a slot was written; Q_out; number of rows without a page)."""
    P, page, n_kv, _ = np.shape(K_codes)
    Qo = None if Q is None else np.array(Q_out, np.float64)
    out = {n: [np.array(c, np.float64), np.array(e, np.int64), np.zeros((P, page), bool)]
           for n, c, e in (("K", K_codes, K_exp), ("V", V_codes, V_exp))}
    entering, lost = {}, 0
    for t, (b, pos) in enumerate(rows_of(q_start, kv_len, len(K))):
        if b < 0 or pos < 0:
            continue
        at = pos + (0 if pos_base is None else int(pos_base[b]))
        if Q is not None:
            Qo[t] = rotated(normed(Q[t], gamma_q, eps), at, inv_freq)
        pg = int(table[b, pos // page]) if pos // page < table.shape[1] else -1
        if not 0 <= pg < P:
            lost += 1
            continue
        entering.setdefault((b, pg), []).append((pos % page, rotated(normed(K[t], gamma_k, eps), at, inv_freq),
                                                 np.asarray(V[t], np.float64)))
    for (b, pg), rows in entering.items():
        first = min(r[0] for r in rows)
        for i, n in enumerate(("K", "V")):
            codes, exps, wrote = out[n]
            for h in range(n_kv):
                e = exponent_for(max(np.abs(r[1 + i][h]).max() for r in rows))
                if first > 0 and exps[pg, h] > e:
                    e = exps[pg, h]
                if first > 0 and exps[pg, h] < e:
                    codes[pg, :first, h] *= 2.0 ** (exps[pg, h] - e)
                    wrote[pg, :first] = True
                exps[pg, h] = e
                for r in rows:
                    codes[pg, r[0], h] = r[1 + i][h] * 2.0 ** -e
                    wrote[pg, r[0]] = True
    return out, Qo, lost


def weight_floor(Q, K_pages, V_codes, V_exp, table, q_start, kv_len, mask_block=0, scale=None):
    """max_j (w_j 2^{v_j}) * sum_j |code_j| of each row, head and dim: what an error in w_j 2^{v_j} of a fixed share of the
    row's largest can come to in the attention's result."""
    Q = np.asarray(Q, np.float64)
    T, n_q, hd = Q.shape
    n_pages, page, n_kv, _ = K_pages.shape
    scale = 1.0 / np.sqrt(hd) if scale is None else scale
    out = np.zeros(Q.shape)
    for t, (b, pos) in enumerate(rows_of(q_start, kv_len, T)):
        if b < 0:
            continue
        end = min(max(0, int(kv_len[b])), table.shape[1] * page)
        if mask_block > 0:
            end = min(end, (pos // mask_block + 1) * mask_block) if pos >= 0 else 0
        j = np.arange(end)
        pg = np.asarray(table[b])[j // page].astype(np.int64)
        j, pg = j[(pg >= 0) & (pg < n_pages)], pg[(pg >= 0) & (pg < n_pages)]
        for h in range(n_q if len(j) else 0):
            g = h // (n_q // n_kv)
            s = np.asarray(K_pages[pg, j % page, g], np.float64) @ Q[t, h] * scale
            w = np.exp(s - s.max())
            out[t, h] = (w / w.sum() * 2.0 ** V_exp[pg, g]).max() * np.abs(V_codes[pg, j % page, g]).sum(0)
    return out


# ---------------------------------------------------------------------------- key weights, eviction
def weights(Q, K_pages, table, q_start, kv_len, lse, score, slot_pos, mask_block=0, scale=None, pos_base=None):
    """-> (score_out, slot_pos_out, magnitude: sum of weight * (1 + |score| + |lse|) of each key), inputs untouched."""
    Q = np.asarray(Q, np.float64)
    T, n_q, hd = Q.shape
    n_pages, page, n_kv, _ = K_pages.shape
    scale = 1.0 / np.sqrt(hd) if scale is None else scale
    out, tag = np.array(score, np.float64), np.array(slot_pos, np.int64)
    mag = np.zeros(out.shape)
    slots = out.shape[2]
    for b in range(len(kv_len)):
        n = int(q_start[b + 1]) - int(q_start[b])
        if n <= 0:
            continue
        L = min(max(0, int(kv_len[b])), table.shape[1] * page, slots)
        first = max(0, int(kv_len[b]) - n)
        if first < L:
            out[b, :, first:L] = 0.0
            tag[b, :, first:L] = np.arange(first, L) + (0 if pos_base is None else int(pos_base[b]))
    for t, (b, pos) in enumerate(rows_of(q_start, kv_len, T)):
        if b < 0:
            continue
        end = min(max(0, int(kv_len[b])), table.shape[1] * page, slots)
        if mask_block > 0:
            end = min(end, (pos // mask_block + 1) * mask_block) if pos >= 0 else 0
        j = np.arange(end)
        pg = np.asarray(table[b])[j // page].astype(np.int64)
        j, pg = j[(pg >= 0) & (pg < n_pages)], pg[(pg >= 0) & (pg < n_pages)]
        for h in range(n_q):
            l = float(lse[t, h])
            if not np.isfinite(l):
                continue
            g = h // (n_q // n_kv)
            s = np.asarray(K_pages[pg, j % page, g], np.float64) @ Q[t, h] * scale
            w = np.exp(s - l)
            out[b, g, j] += w
            mag[b, g, j] += w * (1 + np.abs(s) + abs(l))
    return out, tag, mag


def evict(kv_len, keep, score, slot_pos, recent, pos_base, capacity):
    """-> per (b, g): (K, list of (slot to fill, slot that moves)); capacity: slots that the table and the arrays hold."""
    B, n_kv, slots = np.shape(score)
    out = {}
    for b in range(B):
        L = min(max(0, int(kv_len[b])), capacity, slots)
        K = min(max(0, int(keep[b])), L)
        base = 0 if pos_base is None else int(pos_base[b])
        for g in range(n_kv):
            sc = np.where(np.isnan(score[b, g, :L]), -np.inf, np.asarray(score[b, g, :L], np.float64))
            nan = np.isnan(score[b, g, :L])
            order = sorted(range(L), key=lambda j: (not (recent > 0 and slot_pos[b, g, j] >= L + base - recent), nan[j], -sc[j], j))
            stays = set(order[:K])
            out[b, g] = K, list(zip([j for j in range(K) if j not in stays], sorted(j for j in stays if j >= K)))
    return out


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
