"""Bounds of a decode over the 8-bit cache, per output row, from the arithmetic.

With s_j the score of token j in base 2 (scaled, soft-capped), e_j its V exponent and
code_j its V code, O = sum_j 2^(s_j + e_j) code_j / sum_j 2^s_j. A = the same sum over
|code_j|, from the oracle; M = the row's largest s_j + e_j.
- A score is an fp32 sum of 128 products, truncated by at most 2^-23 of the running sum
  in each of up to 32 additions, and a few more roundings: |ds| <= 2^-18 (1 + scale |q| |k|)
  with the row's own |q|, and a soft-cap c's tanh adds 2^-21 c. LSE moves by no more than
  the largest ds, its logarithm and sum within the same.
- Token weights are f16 values, the largest 2^15, each rounded once: 2^-11 of itself, or,
  below the normal range (2^-14, that is 2^-29 of the largest), 2^-25, that is 2^-40 of the
  largest. A warp's running maximum is at most M, so that a token at or above M - 29 is
  rounded relatively and one below by at most 2^(M - 40).
- O is summed in fp32: 2^-23 of A per product of 16 tokens and per merge of partial states
  (under 64 of them).
- O itself is rounded to bf16: half a step.
"""
import numpy as np

from gpu_helpers import half_ulp_bf16

LOG2E = 1.4426950408889634
U16 = 2.0 ** -11       # relative rounding of a normal f16 value
NORMAL, LAST = 29, 40  # binades below the largest weight: end of the relative rounding, largest error further down


def scores(b, k, ve):
    """Per request: (s [n, H_qo], s + e_v [n, H_qo], pages [n], places [n]) of the visible tokens, base 2, float64.
    k: float64 K values [P, ps, H_kv, 128]; ve: V exponents [P, H_kv]."""
    g, out = b.num_qo_heads // b.num_kv_heads, []
    q = b.q.double().numpy()
    for r in range(b.batch):
        n = int(b.kv_lens[r])
        lo = max(0, n - 1 - b.window_left) if b.window_left > 0 else 0
        tok = np.arange(lo, n)
        page, at = b.kv_indices[b.kv_indptr[r] + tok // b.page_size], tok % b.page_size
        s = np.empty((len(tok), b.num_qo_heads))
        for h in range(b.num_kv_heads):
            s[:, h * g:(h + 1) * g] = k[page, at, h] @ q[r, h * g:(h + 1) * g].T
        s *= b.sm_scale
        if b.soft_cap > 0:
            s = b.soft_cap * np.tanh(s / b.soft_cap)
        s *= LOG2E
        out.append((s, s + np.repeat(ve[page].astype(np.float64), g, 1), page, at))
    return out


def score_error(b, k):
    """ds per row [B, H_qo]."""
    g = b.num_qo_heads // b.num_kv_heads
    qn = np.sqrt((b.q.double().numpy() ** 2).sum(-1))
    kn = np.sqrt((np.nan_to_num(k[np.unique(b.kv_indices)]) ** 2).sum(-1)).max((0, 1), initial=0)
    return 2.0 ** -18 * (1 + b.sm_scale * qn * np.repeat(kn, g)) + 2.0 ** -21 * b.soft_cap


def decode_bounds(b, k, v_codes, ve, O, L, A):
    """(bound of |o - O| [B, H_qo, 128], bound of |lse - L| [B, H_qo]). v_codes: the float64 values of the V codes,
    exponents left out."""
    g = b.num_qo_heads // b.num_kv_heads
    ds = score_error(b, k)
    lost = np.zeros_like(O)
    for r, (s, a, page, at) in enumerate(scores(b, k, ve)):
        if len(s) == 0:
            continue
        M = a.max(0)
        for h in range(b.num_qo_heads):
            small = a[:, h] < M[h] - NORMAL
            if small.any():
                lost[r, h] = 2.0 ** (M[h] - LAST - L[r, h] * LOG2E) * np.abs(v_codes[page[small], at[small], h // g]).sum(0)
    n = int(b.kv_lens.max(initial=0))
    sums = 2.0 ** -23 * (n / 16 + 64)
    bound = half_ulp_bf16(O) * (1 + 2.0 ** -6) + (U16 + 2 * ds[..., None] + sums) * A * (1 + 2.0 ** -7) + lost
    return bound, 2 * ds


def check(o, l, O, L, bound, bound_l):
    """Outputs (o, l) against (O, L) within the bounds; rows without a key hold 0 and -inf."""
    o, l = np.asarray(o, np.float64), np.asarray(l, np.float64)
    empty = np.isneginf(L)
    assert np.array_equal(np.isneginf(l), empty) and np.all(o[empty] == 0) and np.isfinite(o).all()
    excess = (np.abs(o - O) - bound).max(initial=0)
    assert excess <= 0, f"O beyond its bound by {excess}"
    dl = (np.abs(l[~empty] - L[~empty]) - bound_l[~empty]).max(initial=0)
    assert dl <= 0, f"LSE beyond its bound by {dl}"
