"""Plain fp64 restatements of the serving-side operators (test infrastructure; no code shared with the library).

attention: every new row of every request on its own, keys gathered one by one through the page table.
logprobs / logprobs_grad: each row on its own, from the definition of softmax(l / T).
kv_commit: all of a request's reads, then its writes.

Beside each result the oracle reports the magnitudes that bound a correct fp32 computation's rounding.
"""
from __future__ import annotations

import numpy as np

BAD_LAYOUT, TOKEN_RANGE, NONFINITE, SLOT_RANGE = 8, 1, 2, 128


def _slot(table_row, x, page, pages, max_pages):
    """Slot of position x, or -1 outside the cache."""
    if x < 0 or x // page >= max_pages:
        return -1
    p = int(table_row[x // page])
    return p * page + x % page if 0 <= p < pages else -1


def attention(q, k, v, table, seq_lens, row0, rows, scale, row_slots=None, mask=None):
    """q [R, H, D]; k, v [pages, page, G, D]; request b's rows are row0[b] .. row0[b] + rows[b] - 1.

    Returns out [R, H, D], lse [R, H], status [B], and per (row, head) sum p |v| [R, H, D], max_x sum_d |q k| scale and
    the number of keys seen."""
    q, k, v = (np.asarray(a, np.float64) for a in (q, k, v))
    R, H, D = q.shape
    pages, page, G, _ = k.shape
    kf, vf = k.reshape(pages * page, G, D), v.reshape(pages * page, G, D)
    out, lse = np.zeros((R, H, D)), np.full((R, H), -np.inf)
    mag, smax, count = np.zeros((R, H, D)), np.zeros((R, H)), np.zeros(R, np.int64)
    status = np.zeros(len(seq_lens), np.uint32)
    for b, L in enumerate(seq_lens):
        L = int(L)
        if L < 0:
            status[b] |= BAD_LAYOUT
            L = 0
        if L > table.shape[1] * page:
            status[b] |= SLOT_RANGE
            L = table.shape[1] * page
        hist = [_slot(table[b], x, page, pages, table.shape[1]) for x in range(L)]
        new = []
        for j in range(rows[b]):
            if row_slots is None:
                new.append(_slot(table[b], L + j, page, pages, table.shape[1]))
            else:
                s = int(row_slots[row0[b] + j])
                new.append(s if 0 <= s < pages * page else -1)
        if min(hist + new) < 0:
            status[b] |= SLOT_RANGE
        hist = [s for s in hist if s >= 0]
        for i in range(rows[b]):
            sees = [new[j] for j in range(rows[b])
                    if new[j] >= 0 and (j <= i if mask is None else mask[b, i, j] != 0)]
            slots = hist + sees
            r = row0[b] + i
            count[r] = len(slots)
            if not slots:
                continue
            for h in range(H):
                g = h // (H // G)
                kk, vv = kf[slots, g], vf[slots, g]
                with np.errstate(invalid="ignore", over="ignore"):
                    s = kk @ q[r, h] * scale
                    m = s.max()
                    if m == -np.inf:
                        continue
                    e = np.exp(s - m)
                    out[r, h] = (e / e.sum()) @ vv
                    lse[r, h] = m + np.log(e.sum())
                    mag[r, h] = (e / e.sum()) @ np.abs(vv)
                    smax[r, h] = (np.abs(kk) @ np.abs(q[r, h])).max() * abs(scale)
    return {"out": out, "lse": lse, "status": status, "mag": mag, "smax": smax, "count": count}


def kv_commit(cache, table, cu, src, dst, max_len):
    """cache [layers, pages, page, G, D] (one of k, v), moved in a copy; and the requests' status."""
    a = np.array(cache)
    layers, pages, page = a.shape[:3]
    flat = a.reshape(layers, pages * page, *a.shape[3:])
    status = np.zeros(len(cu) - 1, np.uint32)
    for b in range(len(cu) - 1):
        lo, hi = int(cu[b]), int(cu[b + 1])
        if lo < 0 or hi < lo or hi - lo > max_len or hi > len(src):
            status[b] = BAD_LAYOUT
            continue
        moves = []
        for e in range(lo, hi):
            to = _slot(table[b], int(dst[e]), page, pages, table.shape[1])
            if to < 0 or not 0 <= int(src[e]) < pages * page:
                status[b] |= SLOT_RANGE
            else:
                moves.append((to, flat[:, int(src[e])].copy()))
        for to, x in moves:
            flat[:, to] = x
    return a, status


def _temperature(t):
    return float(t) if 1e-30 <= t < np.inf else 1.0


def logprobs(logits, ids, temp=None, top_k=0, row_index=None):
    """logits [rows, V], ids [n, J]: dict of arrays as the library's outputs, plus |l - M| / T weighted by p ("spread")."""
    logits = np.asarray(logits, np.float64)
    rows, V = logits.shape
    n, J = ids.shape
    out = {"logprob": np.zeros((n, J)), "entropy": np.zeros(n), "row_max": np.full(n, -np.inf), "log_z": np.zeros(n),
           "top_ids": np.full((n, top_k), -1, np.int64), "top_logprob": np.full((n, top_k), -np.inf),
           "flags": np.zeros(n, np.uint32), "spread": np.zeros(n)}
    for i in range(n):
        r = i if row_index is None else int(row_index[i])
        if r < 0 or r >= rows:
            out["flags"][i] = 0 if r == -1 else BAD_LAYOUT
            continue
        T = 1.0 if temp is None else _temperature(temp[i])
        l = logits[r].copy()
        bad = np.isnan(l) | (l == np.inf)
        if bad.any():
            out["flags"][i] |= NONFINITE
        l[bad] = -np.inf
        M = l.max()
        lp = np.full(V, -np.inf)
        if M == -np.inf:
            out["flags"][i] |= NONFINITE
            out["log_z"][i] = -np.inf
        else:
            d = (l - M) / T
            Z = np.exp(d).sum()
            lp = d - np.log(Z)
            p = np.exp(lp)
            live = p > 0
            out["row_max"][i], out["log_z"][i] = M, np.log(Z)
            out["entropy"][i] = -(p[live] * lp[live]).sum()
            out["spread"][i] = (p[live] * np.abs(d[live])).sum()
        for j in range(J):
            v = int(ids[i, j])
            if v == -1:
                continue
            if 0 <= v < V:
                out["logprob"][i, j] = lp[v]
            else:
                out["logprob"][i, j] = -np.inf
                out["flags"][i] |= TOKEN_RANGE
        order = np.lexsort((np.arange(V), -l))[:top_k]
        for k, v in enumerate(order):
            if l[v] > -np.inf:
                out["top_ids"][i, k], out["top_logprob"][i, k] = v, lp[v]
    return out


def logprobs_grad(logits, ids, g_logprob, temp=None, g_entropy=None, top_ids=None, g_top=None):
    """dlogits [rows, V] by the formula, and the magnitude of the terms it is the sum of."""
    logits = np.asarray(logits, np.float64)
    rows, V = logits.shape
    d, mag = np.zeros((rows, V)), np.zeros((rows, V))
    for i in range(rows):
        T = 1.0 if temp is None else _temperature(temp[i])
        l = logits[i].copy()
        bad = np.isnan(l) | (l == np.inf)
        l[bad] = -np.inf
        M = l.max()
        if M == -np.inf:
            continue
        x = (l - M) / T
        lp = x - np.log(np.exp(x).sum())
        p = np.exp(lp)
        live = p > 0
        H = -(p[live] * lp[live]).sum()
        terms = [(int(v), float(g)) for v, g in zip(ids[i], g_logprob[i])]
        if g_top is not None:
            terms += [(int(v), float(g)) for v, g in zip(top_ids[i], g_top[i])]
        terms = [(v, g) for v, g in terms if 0 <= v < V and not bad[v]]
        G, A = sum(g for _, g in terms), sum(abs(g) for _, g in terms)
        d[i], mag[i] = -p * G, p * A * (1 + np.where(live, np.abs(lp), 0.0))
        if g_entropy is not None:
            e = np.where(live, p * (np.where(live, lp, 0.0) + H), 0.0)
            d[i] -= g_entropy[i] * e
            mag[i] += abs(g_entropy[i]) * np.where(live, p * (1 + np.abs(np.where(live, lp, 0.0)) + H) ** 2, 0.0)
        for v, g in terms:
            d[i, v] += g
            mag[i, v] += abs(g)
        d[i] /= T
        mag[i] /= T
        d[i][bad] = 0.0
    return d, mag
