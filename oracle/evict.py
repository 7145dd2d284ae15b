"""Plain differential attention, gathered attention weights, the choice of the tokens to
keep and the move of their rows: one request and head at a time, float64.

Rows come as arrays k [P, ps, H, D] of values; a page table as (kv_indptr, kv_indices,
last_page_len). Differential attention splits a row of q and k into two halves, one
softmax map each: o = (P1 - lam P2) v.
"""
from __future__ import annotations

import numpy as np

from . import fp8


def lengths(kv_indptr, last_page_len, ps):
    n = np.diff(np.asarray(kv_indptr, np.int64))
    return np.where(n > 0, (n - 1) * ps + np.asarray(last_page_len, np.int64), 0)


def slots(kv_indptr, kv_indices, b, length, ps):
    """(pages, places) of request b's tokens."""
    t = np.arange(length)
    return np.asarray(kv_indices, np.int64)[int(kv_indptr[b]) + t // ps], t % ps


def scores(q, k, scale, cap, window, n_q, length):
    """Scaled, capped scores [n_q, length] of one head, -inf where the mask hides a key."""
    with np.errstate(invalid="ignore"):
        s = (q @ k.T) * scale
        if cap > 0:
            s = cap * np.tanh(s / cap)
    pos = (length - n_q + np.arange(n_q))[:, None]
    t = np.arange(length)[None, :]
    hidden = t > pos
    if window > 0:
        hidden |= t < pos - window
    return np.where(hidden, -np.inf, s)


def log_sum_exp(s):
    if s.shape[1] == 0:
        return np.full(s.shape[0], -np.inf)
    m = s.max(axis=1)
    ref = np.where(np.isfinite(m), m, 0.0)
    with np.errstate(divide="ignore"):
        return ref + np.log(np.exp(s - ref[:, None]).sum(axis=1))


def differential(q, k, v, qo_indptr, kv_indptr, kv_indices, last_page_len, scale, lam, norm=None, eps=1e-5, out_scale=1.0,
                 window=-1, cap=0.0):
    """(o [n, Hq, D], lse [n, Hq, 2], size [n, Hq, D]); size: what the bound of a rounding error of the weights is
    relative to, (P1 + |lam| P2) |v| before the norm, scaled as the output is."""
    n, Hq, D = q.shape
    ps, H = k.shape[1], k.shape[2]
    g = Hq // H
    o, lse, size = np.zeros((n, Hq, D)), np.full((n, Hq, 2), -np.inf), np.zeros((n, Hq, D))
    for b, L in enumerate(lengths(kv_indptr, last_page_len, ps)):
        q0, q1 = int(qo_indptr[b]), int(qo_indptr[b + 1])
        pg, pl = slots(kv_indptr, kv_indices, b, L, ps)
        for r in range(Hq):
            kk, vv = k[pg, pl, r // g], v[pg, pl, r // g]
            p = []
            for m in range(2):
                half = slice(m * D // 2, (m + 1) * D // 2)
                s = scores(q[q0:q1, r, half], kk[:, half], scale, cap, window, q1 - q0, L)
                z = log_sum_exp(s)
                lse[q0:q1, r, m] = z
                p.append(np.exp(s - np.where(np.isfinite(z), z, 0.0)[:, None]))
            y = (p[0] - lam[r] * p[1]) @ vv
            a = (p[0] + abs(lam[r]) * p[1]) @ np.abs(vv)
            f = np.full((q1 - q0, 1), out_scale)
            if norm is not None:
                f = out_scale / np.sqrt((y * y).mean(axis=1, keepdims=True) + eps) * norm[None, :]
            o[q0:q1, r], size[q0:q1, r] = y * f, a * np.abs(f)
    return o, lse, size


def weights(q, lse, k, w, qo_indptr, kv_indptr, kv_indices, last_page_len, scale, decay=1.0, lam=None, window=-1, cap=0.0):
    """(w after the update, size): size is the sum of the weights' absolute values that went into each entry."""
    n, Hq, D = q.shape
    P, ps, H = k.shape[:3]
    g = Hq // H
    w, size = w.astype(np.float64).copy(), np.zeros(w.shape)
    for b, L in enumerate(lengths(kv_indptr, last_page_len, ps)):
        q0, q1 = int(qo_indptr[b]), int(qo_indptr[b + 1])
        pg, pl = slots(kv_indptr, kv_indices, b, L, ps)
        there = (pg >= 0) & (pg < P)
        pg = np.where(there, pg, 0)
        t = np.arange(L)
        for h in range(H):
            got, mass = np.zeros(L), np.zeros(L)
            for r in range(h * g, (h + 1) * g):
                p = []
                for m in range(1 if lam is None else 2):
                    half = slice(0, D) if lam is None else slice(m * D // 2, (m + 1) * D // 2)
                    s = scores(q[q0:q1, r, half], k[pg, pl, h][:, half], scale, cap, window, q1 - q0, L)
                    z = lse[q0:q1, r] if lam is None else lse[q0:q1, r, m]
                    with np.errstate(invalid="ignore"):
                        x = np.exp(s - z[:, None])
                    p.append(np.where((s == -np.inf) | (z == -np.inf)[:, None], 0.0, x))
                one = p[0] if lam is None else np.abs(p[0] - lam[r] * p[1])
                got += one.sum(axis=0)
                mass += (p[0] if lam is None else p[0] + abs(lam[r]) * p[1]).sum(axis=0)
            old = w[pg, h, pl]
            base = np.where((t < L - (q1 - q0)) & (decay != 0), decay * np.where(decay != 0, old, 0.0), 0.0)
            w[pg[there], h, pl[there]] = (base + got)[there]
            size[pg[there], h, pl[there]] = (np.abs(base) + mass)[there]
    return w, size


def select(w, kv_indptr, kv_indices, last_page_len, budget, max_keep, sinks, recent):
    """(kept [B, H, max_keep], new_lens [B]): a plain sort by (weight descending, position ascending)."""
    P, H, ps = w.shape
    lens = lengths(kv_indptr, last_page_len, ps)
    B = len(lens)
    kept, new = np.full((B, H, max_keep), -1, np.int32), np.zeros(B, np.int32)
    for b, L in enumerate(lens):
        new[b] = min(int(L), max(int(budget[b]), 0), max_keep)
        pg, pl = slots(kv_indptr, kv_indices, b, L, ps)
        there = (pg >= 0) & (pg < P)
        t = np.arange(L)
        for h in range(H):
            x = np.where(there, w[np.where(there, pg, 0), h, pl].astype(np.float64), -np.inf)
            x = np.where(np.isnan(x), -np.inf, x)
            x = np.where((t < sinks) | (t >= L - recent), np.inf, x)
            order = sorted(range(int(L)), key=lambda i: (-x[i], i))
            kept[b, h, :new[b]] = sorted(order[:new[b]])
    return kept, new


def compact(rows, kept, new_lens, kv_indptr, kv_indices, ps):
    """rows [P, ps, H, ...] with the kept tokens moved to the front of their requests (a copy)."""
    out = rows.copy()
    for b in range(len(new_lens)):
        row = np.asarray(kv_indices, np.int64)[int(kv_indptr[b]):int(kv_indptr[b + 1])]
        for h in range(rows.shape[2]):
            for j in range(int(new_lens[b])):
                i = int(kept[b, h, j])
                out[row[j // ps], j % ps, h] = rows[row[i // ps], i % ps, h]
    return out


def compact_codes(codes, exps, kept, new_lens, kv_indptr, kv_indices, ps, encode):
    """The same for e4m3 codes [P, ps, H, D] with exponents [P, H]: (codes, exps)."""
    out, e_out = codes.copy(), exps.copy()
    value = fp8.e4m3_to_float(codes)
    for b in range(len(new_lens)):
        row = np.asarray(kv_indices, np.int64)[int(kv_indptr[b]):int(kv_indptr[b + 1])]
        for h in range(codes.shape[2]):
            for j0 in range(0, int(new_lens[b]), ps):
                js = range(j0, min(j0 + ps, int(new_lens[b])))
                src = [int(kept[b, h, j]) for j in js]
                es = [int(exps[row[i // ps], h]) for i in src]
                e = max(es)
                e_out[row[j0 // ps], h] = e
                for j, i, was in zip(js, src, es):
                    x = value[row[i // ps], i % ps, h]
                    c = codes[row[i // ps], i % ps, h]
                    out[row[j // ps], j % ps, h] = c if was == e else encode(x.astype(np.float64) * 2.0 ** (was - e))
    return out, e_out
