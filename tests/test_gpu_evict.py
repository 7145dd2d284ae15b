"""Gathered attention weights, the choice of the tokens to keep and the move of their rows on the GPU, against the plain
64-bit forms (oracle.evict). The choice and the move are exact; the weights' bound is derived beside `bound`."""
import numpy as np
import pytest
import torch

import workloads
from gpu_helpers import lib
from oracle import evict as ev
from oracle import fp8
from oracle import kv_cache as kc
from test_gpu_fp8_block import cache8

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def bsp():
    return lib()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def table(b):
    return dev(b.kv_indptr.astype(np.int32)), dev(b.kv_indices.astype(np.int32)), dev(b.last_page_len.astype(np.int32))


def values(t):
    return t.double().numpy()


# ---- gathered weights -----------------------------------------------------------
def true_lse(b, k, scale, window, cap, maps):
    n, Hq, D = b.q.shape
    lse, d = np.full((n, Hq, maps), -np.inf), D // maps
    q = values(b.q)
    for i, L in enumerate(ev.lengths(b.kv_indptr, b.last_page_len, b.page_size)):
        q0, q1 = int(b.qo_indptr[i]), int(b.qo_indptr[i + 1])
        pg, pl = ev.slots(b.kv_indptr, b.kv_indices, i, L, b.page_size)
        for r in range(Hq):
            for m in range(maps):
                half = slice(m * d, (m + 1) * d)
                s = ev.scores(q[q0:q1, r, half], k[pg, pl, r // (Hq // k.shape[2])][:, half], scale, cap, window, q1 - q0, L)
                lse[q0:q1, r, m] = ev.log_sum_exp(s)
    return (lse if maps == 2 else lse[:, :, 0]).astype(np.float32)


def bound(b, k, lse, scale, size, cap):
    """|w - w64| for fp32 arithmetic. A score is scale times a sum of D products: off by at most D 2^-23 of scale * sum |q k|
    (tensor cores may cut instead of rounding: 2^-23 per addition), its scaling and the subtraction of LSE by 2^-23 of their
    sizes each, taken times log2 e, and 2^-22 for the exponential; a capped score by 2^-21 cap more (tanh). A weight is off by
    that relatively, and by the additions: 2^-24 per column and 4 more steps."""
    q = np.abs(values(b.q))
    q = np.where(np.isfinite(q), q, 0.0)  # (such a query has LSE -inf and gives nothing)
    big = np.nanmax(np.where(np.isfinite(k), np.abs(k), 0.0))
    s = abs(scale) * q.sum(axis=2).max() * big if q.size else 0.0  # >= scale * sum |q k|
    fin = np.abs(lse[np.isfinite(lse)])
    cols = int(np.diff(b.qo_indptr).max()) * b.q.shape[1] // k.shape[2] if b.q.size else 0
    rel = s * b.q.shape[2] * 2.0 ** -23 + 3 * (s + (fin.max() if fin.size else 0.0)) * 2.0 ** -23 + 2.0 ** -21
    rel += cap * 2.0 ** -21 + (cols + 6) * 2.0 ** -24
    return size * rel


def run_weights(bsp, seed, qo, kv, Hq, H, D, ps, dtype="bf16", f8=False, diff=False, window=-1, cap=0.0, decay=1.0, lse=None,
                qo_none=False, change=None, pad=3, scale=None):
    b = workloads.paged_batch(seed, qo, kv, Hq, H, D, ps, dtype, causal=True, extra_pages=4)
    rng = np.random.default_rng(seed)
    scale = 1 / np.sqrt(D // 2 if diff else D) if scale is None else scale
    ke = None
    if f8:
        codes, e, _, _ = cache8(b, seed)
        k, kt, ke = kc.values(codes, e), dev(codes).view(F8), dev(e)
    else:
        k, kt = values(b.k_pages), b.k_pages.cuda()
    lse = true_lse(b, k, scale, window, cap, 2 if diff else 1) if lse is None else lse
    w = rng.exponential(size=(k.shape[0], H, ps)).astype(np.float32)
    lens = ev.lengths(b.kv_indptr, b.last_page_len, ps)
    for i, L in enumerate(lens):  # what stands in the queries' own slots says nothing
        pg, pl = ev.slots(b.kv_indptr, b.kv_indices, i, L, ps)
        own = np.arange(L) >= L - (int(b.qo_indptr[i + 1]) - int(b.qo_indptr[i]))
        w[pg[own], :, pl[own]] = np.nan
    if change:
        change(b, lse, w)
    lam = (0.8 + 0.1 * rng.standard_normal(Hq)).astype(np.float32) if diff else None
    wt = dev(w)
    indptr, indices, last = table(b)
    indices = torch.cat([indices, torch.full((pad,), -1, dtype=torch.int32, device="cuda")])  # a table with room
    bsp.accumulate_weights(b.q.cuda(), dev(lse), kt, wt, indptr, indices, last,
                           qo_indptr=None if qo_none else dev(b.qo_indptr.astype(np.int32)), sm_scale=scale, decay=decay,
                           k_exp=ke, lam=None if lam is None else dev(lam), window_left=window, logits_soft_cap=cap)
    torch.cuda.synchronize()
    want, size = ev.weights(values(b.q), lse.astype(np.float64), k, w, b.qo_indptr, b.kv_indptr, b.kv_indices, b.last_page_len,
                            scale, decay=decay, lam=lam, window=window, cap=cap)
    got = wt.cpu().numpy().astype(np.float64)
    tol = bound(b, k, lse, scale, size, cap)
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan)
    worst = np.abs(got - want)[~nan] - tol[~nan]
    assert worst.max(initial=-1.0) <= 0, (worst.max(), np.abs(got - want)[~nan].max())
    return b, got, w


DECODE = [  # kv lengths, Hq, H, D, ps
    ([1, 0, 70, 300, 1500], 32, 8, 128, 16), ([64, 63, 65, 128], 8, 8, 128, 1), ([333], 16, 1, 128, 64),
    ([5, 900], 12, 4, 64, 5), ([2000, 1], 40, 2, 128, 12), ([129, 127], 8, 1, 64, 128)]


@pytest.mark.parametrize("case", DECODE, ids=str)
@pytest.mark.parametrize("diff", [False, True], ids=["one", "diff"])
def test_weights_decode_bf16(bsp, case, diff):
    kv, Hq, H, D, ps = case
    run_weights(bsp, 11, [1 if x else 0 for x in kv], kv, Hq, H, D, ps, diff=diff)


@pytest.mark.parametrize("case", DECODE[:3] + [([2000, 1], 40, 2, 128, 12)], ids=str)
@pytest.mark.parametrize("diff", [False, True], ids=["one", "diff"])
def test_weights_decode_e4m3(bsp, case, diff):
    kv, Hq, H, D, ps = case
    run_weights(bsp, 12, [1 if x else 0 for x in kv], kv, Hq, H, D, ps, f8=True, diff=diff, decay=0.97)


@pytest.mark.parametrize("D", [32, 64, 128, 256])
@pytest.mark.parametrize("qo", [1, 7])
def test_weights_f32(bsp, D, qo):
    run_weights(bsp, 13, [qo] * 3, [qo, 200, 77], 6, 2, D, 5, dtype="f32", window=90 if D == 64 else -1, cap=9.0 if D == 128 else 0.0,
                decay=0.5)


@pytest.mark.parametrize("ps", [1, 8, 16, 12, 64, 128])
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "diff", "d64"])
def test_weights_of_prompts(bsp, ps, kind):
    """Whole prompts, chunks behind a cache and observation windows; every query position's mask counts."""
    D = 64 if kind == "d64" else 128
    run_weights(bsp, 14, [300, 1, 64, 33, 0], [300, 1, 515, 34, 40], 16, 4, D, ps, f8=kind == "e4m3", diff=kind == "diff", decay=0.9)


@pytest.mark.parametrize("g", [1, 2, 8, 32])
def test_weights_head_groups(bsp, g):
    run_weights(bsp, 15, [200, 130], [500, 130], 2 * g, 2, 128, 16, decay=0.0)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "diff"])
@pytest.mark.parametrize("window,cap", [(1, 0.0), (50, 0.0), (200, 20.0), (-1, 5.0), (2 ** 31 - 1, 0.0)])
def test_weights_variants(bsp, kind, window, cap):
    run_weights(bsp, 16, [150, 1, 260], [400, 333, 260], 16, 4, 128, 16, f8=kind == "e4m3", diff=kind == "diff", window=window, cap=cap,
                decay=0.0)


def test_weights_of_queries_without_keys(bsp):
    """LSE -inf gives nothing (a sink alone, say); NaN LSE makes NaN of what the query sees, not of the rest."""
    def change(b, lse, w):
        lse[3] = -np.inf
        lse[int(b.qo_indptr[1]), 0] = np.nan
    b, got, _ = run_weights(bsp, 17, [10, 4], [100, 40], 8, 4, 128, 16, change=change)
    pg, pl = ev.slots(b.kv_indptr, b.kv_indices, 1, 40, 16)
    assert np.isnan(got[pg, 0, pl][:37]).all() and not np.isnan(got[pg, 1:, pl][:37]).any()


@pytest.mark.parametrize("kind", ["bf16", "diff"])
@pytest.mark.parametrize("window,cap", [(-1, 0.0), (200, 0.0), (-1, 5.0), (333, 7.0)])
def test_weights_of_long_prompts(bsp, kind, window, cap):
    """From 1024 query rows per request on a unit of keys is a CTA's only one."""
    run_weights(bsp, 23, [600, 520], [700, 520], 8, 2, 128, 16, diff=kind == "diff", window=window, cap=cap, decay=0.5)


@pytest.mark.parametrize("kind", ["bf16", "diff"])
@pytest.mark.parametrize("qo", [[300, 100], [700, 400]], ids=str)
def test_weights_of_prompts_with_strange_queries(bsp, qo, kind):
    """Rows of q that hold NaN or infinities and have LSE -inf, one map's LSE alone, LSE +inf, in full and in partial tiles."""
    def change(b, lse, w):
        for i in (0, 7, 140, 299, 300, 399):
            b.q[i] = float("nan") if i % 2 else float("inf")
            lse[i] = -np.inf
        lse[50, 3] = np.inf
        if kind == "diff":
            lse[60, 2, 0] = lse[70, 5, 1] = -np.inf
    run_weights(bsp, 21, qo, [qo[0], 515], 8, 2, 128, 16, diff=kind == "diff", change=change)


@pytest.mark.parametrize("kind", ["bf16", "diff"])
@pytest.mark.parametrize("scale", [0.0, -0.05, 1e-12, 1e-9, 3e-4, 0.5])
def test_weights_of_prompts_at_any_scale(bsp, scale, kind):
    """LSE enters the products divided by the scale: 24 bits of it, rounded or cut a few times by 2^-23 of its size, which the
    bound's share of LSE and of the columns' additions (hundreds times 2^-24) holds. Scales where that overflows subtract later."""
    run_weights(bsp, 22, [200, 64], [200, 515], 8, 2, 128, 16, diff=kind == "diff", scale=scale, decay=0.5)


def test_weights_without_qo_indptr_and_untouched_rows(bsp):
    b, got, w = run_weights(bsp, 18, [1, 1, 1], [40, 17, 100], 8, 2, 128, 16, qo_none=True)
    used = np.zeros(got.shape, bool)
    for i, L in enumerate([40, 17, 100]):
        pg, pl = ev.slots(b.kv_indptr, b.kv_indices, i, L, 16)
        used[pg, :, pl] = True
    assert np.array_equal(got[~used], w[~used].astype(np.float64), equal_nan=True)


def test_weights_skip_pages_outside_the_pool(bsp):
    def change(b, lse, w):
        b.kv_indices[3] = 1 << 30
        b.kv_indices[5] = -7
    b = workloads.paged_batch(19, [1, 1], [100, 50], 8, 2, 128, 16, "bf16", extra_pages=2)
    k, q = values(b.k_pages), values(b.q)
    lse = true_lse(b, k, 0.1, -1, 0.0, 1)
    w = np.ones((k.shape[0], 2, 16), np.float32)
    change(b, lse, w)
    wt = dev(w)
    bsp.accumulate_weights(b.q.cuda(), dev(lse), b.k_pages.cuda(), wt, *table(b), sm_scale=0.1)
    torch.cuda.synchronize()
    want, size = ev.weights(q, lse.astype(np.float64), k, w, b.qo_indptr, b.kv_indptr, b.kv_indices, b.last_page_len, 0.1)
    assert (np.abs(wt.cpu().numpy() - want) <= bound(b, k, lse, 0.1, size, 0.0)).all()


@pytest.mark.parametrize("qo", [[60, 50], [700, 650]], ids=str)
def test_weights_of_prompts_skip_pages_outside_the_pool(bsp, qo):
    b = workloads.paged_batch(25, qo, [700, 650], 8, 2, 128, 16, "bf16", causal=True, extra_pages=2)
    k, q = values(b.k_pages), values(b.q)
    lse = true_lse(b, k, 0.1, -1, 0.0, 1)
    w = np.ones((k.shape[0], 2, 16), np.float32)
    b.kv_indices[3], b.kv_indices[20:24], b.kv_indices[-1] = 1 << 30, -7, k.shape[0]
    wt = dev(w)
    bsp.accumulate_weights(b.q.cuda(), dev(lse), b.k_pages.cuda(), wt, *table(b), qo_indptr=dev(b.qo_indptr.astype(np.int32)), sm_scale=0.1)
    torch.cuda.synchronize()
    want, size = ev.weights(q, lse.astype(np.float64), k, w, b.qo_indptr, b.kv_indptr, b.kv_indices, b.last_page_len, 0.1)
    assert (np.abs(wt.cpu().numpy() - want) <= bound(b, k, lse, 0.1, size, 0.0)).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "f32", "prompts", "long"])
def test_part_of_a_table(bsp, kind):
    """A slice of the arrays: kv_indptr[0] and qo_indptr[0] are not 0, and what stands before belongs to others."""
    qo = {"prompts": [100, 150, 70], "long": [100, 900, 400]}.get(kind, [1, 1, 1])
    b = workloads.paged_batch(24, qo, [1300, 900, 433], 8, 2, 128, 16, "f32" if kind == "f32" else "bf16", causal=True, extra_pages=2)
    ke = None
    if kind == "e4m3":
        codes, e, _, _ = cache8(b, 24)
        k, kt, ke = kc.values(codes, e), dev(codes).view(F8), dev(e)
    else:
        k, kt = values(b.k_pages), b.k_pages.cuda()
    lse = true_lse(b, k, 0.1, -1, 0.0, 1)
    w = np.random.default_rng(24).exponential(size=(k.shape[0], 2, 16)).astype(np.float32)
    indptr, indices, last = table(b)
    part = indptr[1:].clone(), indices, last[1:].clone()
    wt = dev(w)
    bsp.accumulate_weights(b.q.cuda(), dev(lse), kt, wt, *part, qo_indptr=dev(b.qo_indptr[1:].astype(np.int32)), sm_scale=0.1,
                           decay=0.5, k_exp=ke)
    torch.cuda.synchronize()
    host = b.kv_indptr[1:], b.kv_indices, b.last_page_len[1:]
    want, size = ev.weights(values(b.q), lse.astype(np.float64), k, w, b.qo_indptr[1:], *host, 0.1, decay=0.5)
    got = wt.cpu().numpy()
    assert (np.abs(got - want) <= bound(b, k, lse, 0.1, size, 0.0)).all()
    kept, new = bsp.select_tokens(wt, *part, dev(np.array([300, 100], np.int32)), 300)
    K, N = ev.select(got, *host, np.array([300, 100]), 300, 4, 32)
    assert np.array_equal(kept.cpu().numpy(), K) and np.array_equal(new.cpu().numpy(), N)
    if ke is None:
        v = b.v_pages.cuda()
        bsp.compact_cache(kept, new, *part, kt, v, wt)
        torch.cuda.synchronize()
        kind_ = torch.int32 if kind == "f32" else torch.int16
        for a, g in ((b.k_pages, kt), (b.v_pages, v)):
            moved = ev.compact(a.view(kind_).numpy(), K, N, b.kv_indptr[1:], b.kv_indices, 16)
            assert np.array_equal(g.view(kind_).cpu().numpy(), moved)


def test_weights_of_many_requests(bsp):
    rng = np.random.default_rng(20)
    kv = rng.integers(0, 200, 1500)
    run_weights(bsp, 20, np.minimum(kv, 1), kv, 4, 1, 128, 16)


# ---- tokens to keep ---------------------------------------------------------------
def pool_table(seed, lens, ps, extra=3):
    rng = np.random.default_rng(seed)
    lens = np.asarray(lens, np.int64)
    n = -(-lens // ps)
    ids = rng.permutation(int(n.sum()) + extra).astype(np.int32)
    return (np.concatenate([[0], np.cumsum(n)]).astype(np.int32), ids[:int(n.sum())], np.where(lens > 0, (lens - 1) % ps + 1, 0).astype(np.int32),
            len(ids))


def select(bsp, w, indptr, indices, last, budget, most, sinks, recent, **kw):
    kept, new = bsp.select_tokens(dev(w), dev(indptr), dev(indices), dev(last), dev(np.asarray(budget, np.int32)), most,
                                  sinks=sinks, recent=recent, **kw)
    torch.cuda.synchronize()
    return kept.cpu().numpy(), new.cpu().numpy()


@pytest.mark.parametrize("ps", [1, 5, 16, 128])
@pytest.mark.parametrize("kind", ["spread", "ties", "equal", "odd"])
def test_select(bsp, ps, kind):
    lens = [0, 1, 2, 31, 32, 33, 500, 1029, 2500]
    rng = np.random.default_rng(21)
    indptr, indices, last, P = pool_table(21, lens, ps)
    w = np.exp(3 * rng.standard_normal((P, 3, ps))).astype(np.float32)
    if kind == "ties":
        w = np.floor(w)
    elif kind == "equal":
        w[:] = 0.25
    elif kind == "odd":  # signs, zeros of both signs, infinities, NaN, subnormals
        pick = rng.integers(0, 9, w.shape)
        for i, x in enumerate([0.0, -0.0, np.inf, -np.inf, np.nan, 1e-42, -3.5]):
            w[pick == i] = x
    for budget, most, sinks, recent in [([3, 1, 1, 16, 32, 40, 100, 1000, 1250], 1250, 4, 32), ([0, 0, 1, 1, 5, 33, 499, 1029, 9000], 700, 0, 0),
                                        ([-4, 7, 2, 30, 31, 32, 5, 64, 1], 64, 10, 300)]:
        kept, new = select(bsp, w, indptr, indices, last, budget, most, sinks, recent)
        want, n = ev.select(w, indptr, indices, last, budget, most, sinks, recent)
        assert np.array_equal(new, n) and np.array_equal(kept, want)


@pytest.mark.parametrize("B,H,L,most", [(1, 1, 131072, 4096), (1, 8, 30000, 29999), (2, 2, 100001, 50000), (1, 1, 400000, 777),
                                        (20, 8, 5000, 1), (3, 5, 9000, 9000)])
def test_select_long_rows(bsp, B, H, L, most):
    """Clusters of CTAs, keys that shared memory does not hold, ragged parts: against torch's stable sort."""
    rng = np.random.default_rng(22)
    lens = [L] + [int(x) for x in rng.integers(L // 2, L, B - 1)]
    indptr, indices, last, P = pool_table(22, lens, 16)
    w = np.floor(np.exp(2 * rng.standard_normal((P, H, 16))) * 8).astype(np.float32)
    kept, new = select(bsp, w, indptr, indices, last, [most] * B, most, 4, 64)
    for b, L in enumerate(lens):
        pg, pl = ev.slots(indptr, indices, b, L, 16)
        for h in range(H):
            x = torch.from_numpy(w[pg, h, pl]).clone()
            x[:4] = x[max(0, L - 64):] = np.inf
            n = min(L, most)
            order = torch.sort(x, descending=True, stable=True).indices[:n].sort().values.numpy()
            assert new[b] == n and np.array_equal(kept[b, h, :n], order) and (kept[b, h, n:] == -1).all()


def test_select_outside_pages_and_given_outputs(bsp):
    rng = np.random.default_rng(23)
    indptr, indices, last, P = pool_table(23, [200, 90], 16)
    indices[2], indices[14] = 10 ** 9, -1
    w = rng.standard_normal((P, 2, 16)).astype(np.float32)
    kept, new = (torch.full(s, 77, dtype=torch.int32, device="cuda") for s in ((2, 2, 190), (2,)))
    bsp.select_tokens(dev(w), dev(indptr), dev(indices), dev(last), dev(np.array([150, 50], np.int32)), 190, 0, 3, kept=kept, new_lens=new)
    want, n = ev.select(w, indptr, indices, last, [150, 50], 190, 0, 3)
    assert np.array_equal(new.cpu().numpy(), n) and np.array_equal(kept.cpu().numpy(), want)


# ---- the move -----------------------------------------------------------------
def some_kept(rng, lens, H, most, how):
    kept, new = np.full((len(lens), H, most), -1, np.int32), np.zeros(len(lens), np.int32)
    for b, L in enumerate(lens):
        n = new[b] = min(int(L), int(rng.integers(0, most + 1)) if how != "all" else most)
        for h in range(H):
            if how == "last":
                kept[b, h, :n] = np.arange(L - n, L)
            elif how == "one_gone" and 0 < n < L:
                kept[b, h, :n] = np.delete(np.arange(n + 1), rng.integers(0, n + 1))
            else:
                kept[b, h, :n] = np.sort(rng.permutation(int(L))[:n])
    return kept, new


@pytest.mark.parametrize("ps", [1, 5, 16, 128])
@pytest.mark.parametrize("how", ["random", "last", "one_gone", "all"])
@pytest.mark.parametrize("kind", ["bf16", "bf16_64", "f32", "raw8", "e4m3"])
def test_compact(bsp, ps, how, kind):
    lens, H = [0, 1, 40, 255, 256, 257, 700, 1300], 3
    rng = np.random.default_rng(24)
    indptr, indices, last, P = pool_table(24, lens, ps)
    kept, new = some_kept(rng, lens, H, 900, how)
    w = rng.standard_normal((P, H, ps)).astype(np.float32)
    wt, args = dev(w), (dev(kept), dev(new), dev(indptr), dev(indices), dev(last))
    if kind == "e4m3":
        codes = [rng.integers(0, 256, (P, ps, H, 128)).astype(np.uint8) for _ in range(2)]
        exps = [rng.integers(-20, 3, (P, H)).astype(np.int8) for _ in range(2)]
        kt, vt = (dev(c).view(F8) for c in codes)
        et = [dev(e) for e in exps]
        bsp.compact_cache(*args, kt, vt, weights=wt, k_exp=et[0], v_exp=et[1])
        for c, e, ct, t in zip(codes, exps, (kt, vt), et):
            cw, ew = ev.compact_codes(c, e, kept, new, indptr, indices, ps, kc.encode)
            got = ct.view(torch.uint8).cpu().numpy()
            nan = (cw & 0x7f) == 0x7f  # (a NaN's sign is not kept when it is rescaled)
            assert np.array_equal(t.cpu().numpy(), ew)
            assert np.array_equal(got[~nan], cw[~nan]) and ((got[nan] & 0x7f) == 0x7f).all()
    else:
        D = 64 if kind == "bf16_64" else 128
        dt = {"f32": np.uint32, "raw8": np.uint8}.get(kind, np.uint16)
        rows = [rng.integers(0, np.iinfo(dt).max, (P, ps, H, D)).astype(dt) for _ in range(2)]
        tt = {"f32": torch.float32, "raw8": F8}.get(kind, torch.bfloat16)
        kt, vt = (dev(r.view(np.uint8)).view(tt) for r in rows)
        bsp.compact_cache(*args, kt, vt, weights=wt if how != "last" else None)
        for r, t in zip(rows, (kt, vt)):
            assert np.array_equal(t.view(torch.uint8).cpu().numpy().view(dt), ev.compact(r, kept, new, indptr, indices, ps))
    torch.cuda.synchronize()
    want = ev.compact(np.swapaxes(w, 1, 2), kept, new, indptr, indices, ps).swapaxes(1, 2) if kind == "e4m3" or how != "last" else w
    assert np.array_equal(wt.cpu().numpy(), want)


def test_compact_codes_far_apart(bsp):
    """Every exponent distance from 0 to 255 (below 2^-18 nothing is left of a code), and more rows than one chunk of factors."""
    ps, H, L = 4, 1, 40000
    rng = np.random.default_rng(25)
    indptr, indices, last, P = pool_table(25, [L], ps)
    kept = np.sort(rng.permutation(L)[:36000]).astype(np.int32).reshape(1, 1, -1)
    codes = rng.integers(0, 256, (P, ps, H, 128)).astype(np.uint8)
    exps = rng.integers(-128, 128, (P, H)).astype(np.int8)
    exps[::2] = rng.integers(-20, 1, exps[::2].shape)
    kt, vt, ke, ve = dev(codes).view(F8), dev(codes[::-1]).view(F8), dev(exps), dev(exps[::-1])
    bsp.compact_cache(dev(kept), dev(np.array([36000], np.int32)), dev(indptr), dev(indices), dev(last), kt, vt, k_exp=ke, v_exp=ve)
    torch.cuda.synchronize()
    row = indices.astype(np.int64)
    src, j = kept[0, 0].astype(np.int64), np.arange(36000)
    for c, e, t, et in ((codes, exps, kt, ke), (codes[::-1], exps[::-1], vt, ve)):
        es = e[row[src // ps], 0].astype(int)
        top = np.repeat(np.maximum.reduceat(es, np.arange(0, 36000, ps)), ps)
        assert np.array_equal(et.cpu().numpy()[row[j // ps], 0], top)
        x, was = fp8.e4m3_to_float(c[row[src // ps], src % ps, 0]), c[row[src // ps], src % ps, 0]
        want = np.where((top == es)[:, None], was, kc.encode(x.astype(np.float64) * 2.0 ** (es - top)[:, None]))
        got = t.view(torch.uint8).cpu().numpy()[row[j // ps], j % ps, 0]
        nan = (want & 0x7f) == 0x7f
        assert np.array_equal(got[~nan], want[~nan]) and ((got[nan] & 0x7f) == 0x7f).all()


def test_compact_malformed_lists_stay_inside(bsp):
    """Entries below their place, behind the request or of pages outside the pool move nothing; other requests' rows stay."""
    ps, H = 16, 2
    rng = np.random.default_rng(26)
    indptr, indices, last, P = pool_table(26, [100, 64], ps)
    rows = rng.standard_normal((P, ps, H, 128)).astype(np.float32)
    kept = np.sort(rng.integers(0, 100, (2, H, 40)), axis=2).astype(np.int32)
    kept[0, 0, 5], kept[0, 1, 7], kept[1, :, :] = -1, 10 ** 9, 10 ** 8
    k, v = dev(rows), dev(rows)
    bsp.compact_cache(dev(kept), dev(np.array([40, 900], np.int32)), dev(indptr), dev(indices), dev(last), k, v)
    torch.cuda.synchronize()
    got = k.cpu().numpy()
    assert torch.equal(k, v)
    row = indices.astype(np.int64)
    assert np.array_equal(got[row[indptr[1]:]], rows[row[indptr[1]:]])
    assert np.array_equal(got[row[0], 5, 0], rows[row[0], 5, 0]) and np.array_equal(got[row[0], 7, 1], rows[row[0], 7, 1])


# ---- the calls together, on streams and in graphs ------------------------------------
def test_refusals_of_the_binding(bsp):
    q, lse = torch.zeros(2, 8, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, 8, device="cuda")
    k, w = torch.zeros(3, 16, 2, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(3, 2, 16, device="cuda")
    t = (torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda"), torch.tensor([0, 1], dtype=torch.int32, device="cuda"),
         torch.tensor([3, 4], dtype=torch.int32, device="cuda"))
    ok = dict(q=q, lse=lse, k_pages=k, weights=w, kv_indptr=t[0], kv_indices=t[1], last_page_len=t[2])
    bsp.accumulate_weights(**ok)
    for bad in (dict(q=q.half()), dict(q=q[:, :7]), dict(lse=lse[:1]), dict(lse=lse.double()), dict(k_pages=k.float()), dict(weights=w[:2]),
                dict(weights=w.transpose(1, 2)), dict(kv_indptr=t[0].long()), dict(last_page_len=t[2][:1]), dict(q=q[:1], lse=lse[:1]),
                dict(k_exp=torch.zeros(3, 2, dtype=torch.int8, device="cuda")), dict(lam=torch.ones(8, device="cuda")), dict(kv_indices=t[1].cpu()),
                dict(qo_indptr=t[0][:2]), dict(q=q.transpose(0, 1).contiguous().transpose(0, 1))):
        with pytest.raises(ValueError):
            bsp.accumulate_weights(**{**ok, **bad})
    budget = torch.tensor([2, 2], dtype=torch.int32, device="cuda")
    kept, new = bsp.select_tokens(w, *t, budget, 2)
    for bad in (dict(max_keep=-1), dict(budget=budget[:1]), dict(weights=w.double()), dict(kept=kept[:1]), dict(new_lens=new.long())):
        with pytest.raises(ValueError):
            bsp.select_tokens(**{**dict(weights=w, kv_indptr=t[0], kv_indices=t[1], last_page_len=t[2], budget=budget, max_keep=2), **bad})
    with pytest.raises(bsp.BspError):
        bsp.select_tokens(w, *t, budget, 2, sinks=-1)
    c = dict(kept=kept, new_lens=new, kv_indptr=t[0], kv_indices=t[1], last_page_len=t[2], k_pages=k, v_pages=k.clone())
    bsp.compact_cache(**c)
    for bad in (dict(kept=kept[:, :1]), dict(new_lens=new[:1]), dict(v_pages=k[:2]), dict(v_pages=k.float()), dict(weights=w[:1]),
                dict(k_exp=torch.zeros(3, 2, dtype=torch.int8, device="cuda")), dict(k_pages=k.transpose(1, 2).contiguous().transpose(1, 2))):
        with pytest.raises(ValueError):
            bsp.compact_cache(**{**c, **bad})


def test_empty_batches(bsp):
    i32 = torch.int32
    z = lambda *s, d=i32: torch.zeros(s, dtype=d, device="cuda")  # noqa: E731
    w, k = z(2, 2, 16, d=torch.float32), z(2, 16, 2, 128, d=torch.bfloat16)
    bsp.accumulate_weights(z(0, 8, 128, d=torch.bfloat16), z(0, 8, d=torch.float32), k, w, z(1), z(0), z(0), qo_indptr=z(1))
    kept, new = bsp.select_tokens(w, z(1), z(0), z(0), z(0), 5)
    assert kept.shape == (0, 2, 5) and new.shape == (0,)
    kept, new = bsp.select_tokens(w, z(3), z(0), z(2), z(2) + 4, 5)
    assert (kept == -1).all() and (new == 0).all()
    bsp.compact_cache(kept, new, z(3), z(0), z(2), k, k.clone(), weights=w)
    bsp.compact_cache(kept[:0], new[:0], z(1), z(0), z(0), k, k.clone())
    torch.cuda.synchronize()


def serving_step(bsp, kind):
    """A decode over a cache, its weights, the choice and the move: (buffers, step, the plan's object)."""
    rng = np.random.default_rng(30)
    kv = np.array([500, 33, 260, 1])
    b = workloads.paged_batch(30, np.ones(4, int), kv, 16, 4, 128, 16, "bf16", extra_pages=2)
    lens = torch.tensor([250, 40, 100, 9], dtype=torch.int32, device="cuda")
    ke = ve = None
    if kind == "e4m3":
        k8, ke, v8, ve = (dev(x) for x in cache8(b, 30))
        k, v = k8.view(F8), v8.view(F8)
    else:
        k, v = b.k_pages.cuda(), b.v_pages.cuda()
    s = dict(q=b.q.cuda(), k=k, v=v, ke=ke, ve=ve, w=dev(rng.exponential(size=(k.shape[0], 4, 16)).astype(np.float32)), budget=lens,
             kept=torch.zeros(4, 4, 250, dtype=torch.int32, device="cuda"), new=torch.zeros(4, dtype=torch.int32, device="cuda"))
    t = table(b)
    pa = bsp.PagedAttention("decode", 16, 4, 128, 16, max_batch=4)
    pa.plan(b.kv_indptr, b.last_page_len)
    s["o"], s["lse"] = torch.zeros_like(s["q"]), torch.zeros(4, 16, device="cuda")

    def step(stream=None):
        pa.run(s["q"], k, v, t[1], out=s["o"], lse=s["lse"], k_exp=ke, v_exp=ve, stream=stream)
        bsp.accumulate_weights(s["q"], s["lse"], k, s["w"], *t, decay=0.9, k_exp=ke, stream=stream)
        bsp.select_tokens(s["w"], *t, s["budget"], 250, 4, 8, kept=s["kept"], new_lens=s["new"], stream=stream)
        bsp.compact_cache(s["kept"], s["new"], *t, k, v, weights=s["w"], k_exp=ke, v_exp=ve, stream=stream)
    return s, step, pa, b


def bits(s):
    return [x.clone().view(torch.uint8) for x in (s["o"], s["lse"], s["w"], s["kept"], s["new"], s["k"], s["v"]) + ((s["ke"], s["ve"]) if s["ke"] is not None else ())]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_step_together(bsp, kind):
    """Attention after the eviction is attention over the kept tokens; a captured step replays as the plain one, and the
    step on another stream gives the same bits."""
    s, step, pa, b = serving_step(bsp, kind)
    step()
    torch.cuda.synchronize()
    want = bits(s)
    # the plain forms, from the GPU's own LSE and weights on
    s2, step2, _, _ = serving_step(bsp, kind)
    k = kc.values(s2["k"].view(torch.uint8).cpu().numpy(), s2["ke"].cpu().numpy()) if kind == "e4m3" else values(s2["k"].cpu())
    v = kc.values(s2["v"].view(torch.uint8).cpu().numpy(), s2["ve"].cpu().numpy()) if kind == "e4m3" else values(s2["v"].cpu())
    kept, new = s["kept"].cpu().numpy(), s["new"].cpu().numpy()
    assert new.tolist() == [250, 33, 100, 1]
    lens = ev.lengths(b.kv_indptr, b.last_page_len, 16)
    after = bsp.PagedAttention("decode", 16, 4, 128, 16, max_batch=4)
    n_pages = -(-new // 16)
    indices = np.concatenate([b.kv_indices[b.kv_indptr[i]:b.kv_indptr[i] + n_pages[i]] for i in range(4)]).astype(np.int32)
    after.plan(np.concatenate([[0], np.cumsum(n_pages)]), (new - 1) % 16 + 1)
    o, lse = after.run(s["q"], s["k"], s["v"], dev(indices), k_exp=s["ke"], v_exp=s["ve"])
    q = values(s["q"].cpu())
    for i in range(4):
        pg, pl = ev.slots(b.kv_indptr, b.kv_indices, i, lens[i], 16)
        for r in range(16):
            at = kept[i, r // 4, :new[i]]
            x = (k[pg, pl, r // 4][at] @ q[i, r]) * 128 ** -0.5
            z = np.log(np.exp(x - x.max()).sum()) + x.max()
            y = np.exp(x - z) @ v[pg, pl, r // 4][at]
            # e4m3: a code that moved into a page of a larger exponent was rounded, by up to 2^-4 of its value
            tol = (1e-2, 1e-3) if kind == "bf16" else (None, None)
            if tol[0]:
                assert abs(lse[i, r].item() - z) <= tol[1] and np.abs(o[i, r].double().cpu().numpy() - y).max() <= tol[0] + 2.0 ** -8 * np.abs(y).max()
    # another stream
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    step2(st)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(bits(s2), want))
    # captured and replayed
    s3, step3, _, _ = serving_step(bsp, kind)
    first = [x.clone() for x in (s3["k"].view(torch.uint8), s3["v"].view(torch.uint8), s3["w"])]
    exps = [s3[e].clone() for e in ("ke", "ve") if s3[e] is not None]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step3()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step3()
    for _ in range(2):
        for x, y in zip((s3["k"].view(torch.uint8), s3["v"].view(torch.uint8), s3["w"]), first):
            x.copy_(y)
        for e, y in zip(("ke", "ve"), exps):
            s3[e].copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(bits(s3), want))
