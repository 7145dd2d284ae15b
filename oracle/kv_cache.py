"""Plain 8-bit KV cache: page tables from lengths and the quantising append, one
element at a time where it matters, in float64 and whole numbers.

Codes are e4m3 (oracle.fp8), one exponent per (page, kv head): value = code *
2^exp, exp in [EXP_MIN, EXP_MAX].
"""
from __future__ import annotations

import numpy as np

from . import fp8

EXP_MIN, EXP_MAX = -117, 119
_POSITIVE = np.array([fp8.e4m3_value(c) for c in range(0x7f)])  # 0 .. 448, ascending


def encode(x: np.ndarray) -> np.ndarray:
    """Nearest e4m3 code of float64 values (ties to the even code), saturated at
    448; infinities and NaN give the NaN code 0x7f."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(x), 448.0)
    fin = np.isfinite(x)
    a = np.where(fin, a, 0.0)
    hi = np.clip(np.searchsorted(_POSITIVE, a), 1, 126)  # _POSITIVE[hi - 1] < a <= _POSITIVE[hi]
    lo = hi - 1
    up, down = _POSITIVE[hi] - a, a - _POSITIVE[lo]
    code = np.where(up < down, hi, np.where(down < up, lo, np.where(hi % 2 == 0, hi, lo)))
    code = np.where(a == 0, 0, code).astype(np.uint8)
    code = np.where(np.signbit(x), code | 0x80, code)
    return np.where(fin, code, 0x7f).astype(np.uint8)


def exponent_for(amax: float) -> int:
    """Least e in [EXP_MIN, EXP_MAX] with amax <= 448 * 2^e (EXP_MAX if none)."""
    for e in range(EXP_MIN, EXP_MAX):
        if amax <= 448.0 * 2.0 ** e:
            return e
    return EXP_MAX


def append(x: np.ndarray, slots, codes: np.ndarray, exps: np.ndarray):
    """Append x [n, H, D] (float64) through slots into copies of codes [P, ps, H, D]
    (uint8) and exps [P, H] (int8); returns (codes, exps)."""
    codes, exps = codes.copy(), exps.copy()
    P, ps = codes.shape[:2]
    slots = [int(s) for s in slots]
    i, n = 0, len(slots)
    while i < n:
        if not 0 <= slots[i] < P * ps:
            i += 1
            continue
        page, j = slots[i] // ps, i
        while j < n and 0 <= slots[j] < P * ps and slots[j] // ps == page:
            j += 1
        first = slots[i] % ps
        for h in range(x.shape[1]):
            part = x[i:j, h]
            fin = np.abs(part[np.isfinite(part)])
            e = exponent_for(float(fin.max()) if fin.size else 0.0)
            if first > 0:
                had = int(exps[page, h])
                e = max(e, had)
                if e > had:
                    codes[page, :first, h] = encode(fp8.dequantize(codes[page, :first, h], 1.0) * 2.0 ** (had - e))
            exps[page, h] = e
            for t in range(i, j):
                codes[page, slots[t] % ps, h] = encode(x[t, h] * 2.0 ** -e)
        i = j
    return codes, exps


def values(codes: np.ndarray, exps: np.ndarray) -> np.ndarray:
    """float64 values of a cache [P, ps, H, D]."""
    return fp8.dequantize(codes, 1.0) * np.exp2(exps.astype(np.float64))[:, None, :, None]


def tables(cached, new, free, num_free, block_table, page_size, max_table_pages, max_new_tokens):
    """The outputs of one step, as a dict (block_table a grown copy)."""
    B, width = block_table.shape
    bt = block_table.copy()
    kv_indptr, qo_indptr, last, indices, slots, pos = [0], [0], [], [], [], []
    flags, wanted = 0, 0
    free = [int(f) for f in free][:max(0, min(int(num_free), len(free)))]
    for b in range(B):
        c, m = int(cached[b]), int(new[b])
        if c < 0 or m < 0:
            flags |= 4
        c, m = max(c, 0), max(m, 0)
        want = -(-(c + m) // page_size)
        if want > width:
            flags |= 2
        pages = min(want, width)
        for i in range(min(-(-c // page_size), pages), pages):
            bt[b, i] = free[wanted] if wanted < len(free) else -1
            wanted += 1
        indices += [max(0, int(p)) for p in bt[b, :pages]]
        kv_indptr.append(kv_indptr[-1] + pages)
        qo_indptr.append(qo_indptr[-1] + m)
        last.append((min(c + m, pages * page_size) - 1) % page_size + 1 if pages else 0)
        for t in range(c, c + m):
            if len(slots) >= max_new_tokens:
                break
            p = int(bt[b, t // page_size]) if t // page_size < pages else -1
            slots.append(p * page_size + t % page_size if p >= 0 else -1)
            pos.append(t)
    if wanted > len(free):
        flags |= 1
    if kv_indptr[-1] > max_table_pages or qo_indptr[-1] > max_new_tokens:
        flags |= 2
    indices = (indices + [0] * max_table_pages)[:max_table_pages]
    slots = (slots + [-1] * max_new_tokens)[:max_new_tokens]
    pos = (pos + [0] * max_new_tokens)[:max_new_tokens]
    i32 = lambda a: np.array(a, np.int32)  # noqa: E731
    return {"block_table": bt, "kv_indptr": i32(kv_indptr), "last_page_len": i32(last), "kv_indices": i32(indices),
            "qo_indptr": i32(qo_indptr), "slot_map": np.array(slots, np.int64), "positions": i32(pos),
            "counts": i32([kv_indptr[-1], qo_indptr[-1], min(wanted, len(free)), flags])}
