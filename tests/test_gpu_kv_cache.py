"""Page tables and the quantising append on the GPU against the oracle's plain
forms (oracle.kv_cache). Both are exact: whole numbers, and codes that are one
rounding of an exactly scaled value, so every comparison is for equality."""
import numpy as np
import pytest
import torch

from gpu_helpers import lib
from oracle import kv_cache as kc

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bsp():
    return lib()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


# ---- tables --------------------------------------------------------------------
def make_tables(rng, B, ps, hi, new_hi, width=None, short=0):
    cached = rng.integers(0, hi + 1, B).astype(np.int32)
    new = rng.integers(0, new_hi + 1, B).astype(np.int32)
    if B > 2:
        cached[1], new[1] = 0, 0
    old, tot = -(-cached.astype(np.int64) // ps), -(-(cached.astype(np.int64) + new) // ps)
    width = width or max(1, int(tot.max()) + 2)
    ids = rng.permutation(int(tot.sum()) + 9).astype(np.int32)
    bt = np.full((B, width), -1, np.int32)
    k = 0
    for b in range(B):
        n = min(int(old[b]), width)
        bt[b, :n] = ids[k:k + n]
        k += n
    free = ids[k:]
    need = int((np.minimum(tot, width) - np.minimum(old, width)).sum())
    return cached, new, free, max(0, need - short) if short else len(free), bt


def run_tables(bsp, cached, new, free, nfree, bt, ps, cap_p, cap_t, view=False):
    if view:  # a table that is a window of a wider one
        big = torch.full((bt.shape[0], bt.shape[1] + 5), -7, dtype=torch.int32, device="cuda")
        t = big[:, 2:2 + bt.shape[1]]
        t.copy_(dev(bt))
    else:
        t = dev(bt)
    out = bsp.build_page_tables(dev(cached), dev(new), dev(free), dev(np.array([nfree], np.int32)), t, ps, cap_p, cap_t)
    torch.cuda.synchronize()
    got = {f: getattr(out, f).cpu().numpy() for f in out._fields}
    got["block_table"] = t.cpu().numpy()
    if view:
        assert (big[:, :2] == -7).all() and (big[:, 2 + bt.shape[1]:] == -7).all()
    return got


def same(got, want):
    for f, w in want.items():
        assert np.array_equal(got[f], w), (f, got[f][:20], w[:20])


@pytest.mark.parametrize("seed,B,ps,hi,new_hi,pad", [
    (1, 1, 16, 0, 1, 0), (2, 1, 1, 5, 3, 3), (3, 7, 5, 40, 1, 0), (4, 300, 16, 900, 1, 64), (5, 33, 1, 200, 90, 1),
    (6, 64, 128, 5000, 700, 0), (7, 5, 16, 0, 0, 4), (8, 2000, 8, 60, 20, 5), (9, 9000, 4, 5, 2, 0)])
def test_tables(bsp, seed, B, ps, hi, new_hi, pad):
    rng = np.random.default_rng(seed)
    a = make_tables(rng, B, ps, hi, new_hi)
    tot = int((-(-(a[0].astype(np.int64) + a[1]) // ps)).sum())
    cp, ct = tot + pad, int(a[1].sum()) + pad
    same(run_tables(bsp, *a, ps, cp, ct, view=seed % 2 == 0), kc.tables(*a, ps, cp, ct))


@pytest.mark.parametrize("kind", ["short", "no_free", "narrow", "few_entries", "few_slots", "negative", "bad_num_free"])
def test_tables_that_do_not_fit(bsp, kind):
    rng = np.random.default_rng(20)
    B, ps = 12, 4
    cached, new, free, nfree, bt = make_tables(rng, B, ps, 50, 30, width=9 if kind == "narrow" else None,
                                               short=3 if kind == "short" else 0)
    cp, ct = 400, 400
    if kind == "no_free":
        free, nfree = free[:0], 0
    if kind == "few_entries":
        cp = 11
    if kind == "few_slots":
        ct = 13
    if kind == "negative":
        cached[2], new[5] = -3, -1
    if kind == "bad_num_free":
        nfree = 1 << 30  # more than the list holds
    got, want = run_tables(bsp, cached, new, free, nfree, bt, ps, cp, ct), \
        kc.tables(cached, new, free, nfree, bt, ps, cp, ct)
    same(got, want)
    bit = {"short": 1, "no_free": 1, "narrow": 2, "few_entries": 2, "few_slots": 2, "negative": 4, "bad_num_free": 0}
    assert got["counts"][3] & 7 == bit[kind] or kind in ("no_free", "narrow") and got["counts"][3] & bit[kind]


def test_tables_empty_batch(bsp):
    z = np.zeros(0, np.int32)
    bt = np.zeros((0, 4), np.int32)
    same(run_tables(bsp, z, z, z, 0, bt, 16, 5, 6), kc.tables(z, z, z, 0, bt, 16, 5, 6))


def test_tables_huge_lengths_saturate(bsp):
    """Token sums past int32: the error bit, and nothing out of bounds."""
    cached = np.array([2 ** 31 - 5, 10], np.int32)
    new = np.array([2 ** 31 - 1, 2 ** 31 - 1], np.int32)
    bt = np.full((2, 3), 1, np.int32)
    got = run_tables(bsp, cached, new, np.arange(4, dtype=np.int32), 4, bt, 16, 8, 8)
    assert got["counts"].tolist() == [6, 2 ** 31 - 1, 2, 2]
    assert got["slot_map"].tolist() == [-1] * 8 and got["kv_indptr"].tolist() == [0, 3, 6]


def test_tables_single_token_pages_past_31_bits(bsp):
    """Columns of new tokens from 2^31 on, far past the row: no slot."""
    cached, new = np.array([2 ** 31 - 1, 2 ** 31 - 2], np.int32), np.array([5, 3], np.int32)
    bt = np.full((2, 3), 1, np.int32)
    got = run_tables(bsp, cached, new, np.arange(4, dtype=np.int32), 4, bt, 1, 8, 10)
    assert got["counts"].tolist() == [6, 8, 0, 2]
    assert got["slot_map"].tolist() == [-1] * 10 and got["qo_indptr"].tolist() == [0, 5, 8]
    assert got["positions"].tolist() == [2 ** 31 - 1] * 5 + [2 ** 31 - 2] + [2 ** 31 - 1] * 2 + [0, 0]
    assert (got["block_table"] == 1).all()


# ---- append --------------------------------------------------------------------
def make_cache(rng, P, ps, H):
    codes = rng.integers(0, 256, (P, ps, H, 128)).astype(np.uint8)
    exps = rng.integers(-12, 4, (P, H)).astype(np.int8)
    return codes, exps


def make_slots(rng, P, ps, cached, new):
    perm = rng.permutation(P)
    slots, k = [], 0
    for c, m in zip(cached, new):
        n = -(-(c + m) // ps)
        pages = perm[k:k + n]
        k += n
        slots += [int(pages[t // ps]) * ps + t % ps for t in range(c, c + m)]
    assert k <= P
    return np.array(slots, np.int64)


def run_append(bsp, xk, xv, slots, kc_, vc_, layout="plain", stream=None, times=1):
    (k8, ke), (v8, ve) = kc_, vc_
    f8 = torch.float8_e4m3fn
    t = [dev(k8).view(f8), dev(v8).view(f8), dev(ke), dev(ve)]
    n, H, D = xk.shape
    if layout == "plain":
        k, v = xk.cuda(), xv.cuda()
    elif layout == "fused":  # slices of one projection
        both = torch.cat([torch.zeros(n, 3 * D, dtype=xk.dtype), xk.reshape(n, -1), xv.reshape(n, -1)], 1).cuda()
        k, v = both[:, 3 * D:(3 + H) * D].unflatten(1, (H, D)), both[:, (3 + H) * D:].unflatten(1, (H, D))
    else:  # heads outside tokens
        k, v = (x.permute(1, 0, 2).contiguous().cuda().permute(1, 0, 2) for x in (xk, xv))
    for _ in range(times):
        bsp.append_kv(k, v, dev(slots), *t, stream=stream)
    torch.cuda.synchronize()
    return [t[0].view(torch.uint8).cpu().numpy(), t[2].cpu().numpy(), t[1].view(torch.uint8).cpu().numpy(),
            t[3].cpu().numpy()]


def check_append(got, xk, xv, slots, kc_, vc_):
    nan = lambda c: np.where(c & 0x7f == 0x7f, 0x7f, c)  # noqa: E731  (one NaN)
    for x, (c0, e0), (c, e) in ((xk, kc_, got[:2]), (xv, vc_, got[2:])):
        wc, we = kc.append(x.double().numpy(), slots, c0, e0)
        assert np.array_equal(e, we)
        assert np.array_equal(nan(c), nan(wc))
        untouched = np.ones(c0.shape[0], bool)
        untouched[[s // c0.shape[1] for s in slots if 0 <= s < c0.shape[0] * c0.shape[1]]] = False
        assert np.array_equal(c[untouched], c0[untouched])


def values(rng, n, H, dtype):
    x = rng.standard_normal((n, H, 128)) * np.exp2(rng.uniform(-6, 6, (n, H, 1)))
    return torch.from_numpy(x).to(dtype)


CASES = [  # (seed, ps, H, cached, new, dtype, layout)
    (1, 16, 2, [0], [1], torch.bfloat16, "plain"),
    (2, 16, 8, [3, 15, 16, 0, 31], [1, 1, 1, 1, 1], torch.bfloat16, "fused"),         # a decode step
    (3, 16, 2, [5, 0, 40], [70, 133, 16], torch.bfloat16, "heads"),                    # runs across windows
    (4, 1, 3, [4, 0], [150, 9], torch.bfloat16, "plain"),                              # a page per token
    (5, 5, 1, [2, 7], [131, 300], torch.float32, "fused"),                             # odd pages
    (6, 64, 2, [60, 1], [200, 130], torch.float32, "heads"),
    (7, 128, 1, [0, 100], [400, 200], torch.bfloat16, "plain"),
    (8, 300, 2, [0, 250], [700, 411], torch.bfloat16, "plain"),                        # a page over several windows
    (9, 8, 5, [0] * 40, [1] * 40, torch.float32, "plain"),
    (10, 1000, 1, [13], [900], torch.float32, "plain"),
    # runs of a warp: pages of 2 to 16 tokens, gaps of all lengths, fp32 into larger pages with many runs
    (11, 2, 3, [1, 0, 5] * 9, [1, 7, 4] * 9, torch.bfloat16, "heads"),
    (12, 16, 1, list(range(17)) * 3, list(range(1, 52)), torch.bfloat16, "plain"),
    (13, 7, 2, [3] * 30, [1, 20, 6] * 10, torch.float32, "fused"),
    (14, 15, 1, [14, 15, 16], [47, 31, 500], torch.bfloat16, "plain"),
    (16, 33, 16, [5, 0], [2000, 3001], torch.float32, "fused"),
    (17, 40, 16, [7, 0], [1800, 2100], torch.bfloat16, "heads"),
]


@pytest.mark.parametrize("case", CASES, ids=[f"append{c[0]}" for c in CASES])
def test_append(bsp, case):
    seed, ps, H, cached, new, dtype, layout = case
    rng = np.random.default_rng(seed)
    P = sum(-(-(c + m) // ps) for c, m in zip(cached, new)) + 3
    n = sum(new)
    xk, xv = values(rng, n, H, dtype), values(rng, n, H, dtype)
    slots = make_slots(rng, P, ps, cached, new)
    kc_, vc_ = make_cache(rng, P, ps, H), make_cache(rng, P, ps, H)
    check_append(run_append(bsp, xk, xv, slots, kc_, vc_, layout), xk, xv, slots, kc_, vc_)
    again = run_append(bsp, xk, xv, slots, kc_, vc_, layout, times=2)  # the same tokens twice: the same cache
    check_append(again, xk, xv, slots, kc_, vc_)


def test_append_special_values(bsp):
    """Infinities, NaN, zeros, subnormals, saturation, values at and next to a border of the exponent."""
    rng = np.random.default_rng(30)
    n, H, ps = 24, 2, 4
    x = rng.standard_normal((n, H, 128))
    x[0, 0, 3], x[1, 1, 5], x[2, 0] = np.inf, np.nan, np.nan
    x[4:8] = 0.0
    x[8:12] *= 2.0 ** -130
    x[12:14] *= 2.0 ** 124
    x[16:20] = 0.0
    x[16, 0, 0], x[17, 1, 0] = 448.0 * 2.0 ** -6, np.nextafter(np.float32(448.0), np.float32(500.0)) * 2.0 ** -6
    for dtype in (torch.float32, torch.bfloat16):
        xk = torch.from_numpy(x).to(dtype)
        xv = -xk
        slots = make_slots(rng, 9, ps, [0], [n])
        kc_, vc_ = make_cache(rng, 9, ps, H), make_cache(rng, 9, ps, H)
        check_append(run_append(bsp, xk, xv, slots, kc_, vc_), xk, xv, slots, kc_, vc_)


@pytest.mark.parametrize("ps,n", [(1, 40), (4, 100), (100, 150), (300, 290)])
def test_append_infinities_and_nan_anywhere(bsp, ps, n):
    """Either sign, next to each other and to finite values, whole rows of them: they become NaN and count for nothing."""
    rng = np.random.default_rng(50 + ps)
    H = 2
    x = rng.standard_normal((n, H, 128)) * np.exp2(rng.uniform(-6, 6, (n, H, 1)))
    for bad in (np.inf, -np.inf, np.nan):
        x[rng.random(x.shape) < 0.02] = bad
        x[rng.integers(0, n, 3), 1] = bad
        x[rng.integers(0, n), 0, 8:24] = bad
    P = -(-n // ps) + 2
    for dtype in (torch.float32, torch.bfloat16):
        xk = torch.from_numpy(x).to(dtype)
        xv = xk.flip(0)
        slots = make_slots(rng, P, ps, [0], [n])
        kc_, vc_ = make_cache(rng, P, ps, H), make_cache(rng, P, ps, H)
        check_append(run_append(bsp, xk, xv, slots, kc_, vc_), xk, xv, slots, kc_, vc_)


def test_append_skips_slots_outside_the_pool(bsp):
    """A padded step: slots of -1 at the end (and past the pool), an unused window in the middle of a page."""
    rng = np.random.default_rng(31)
    n, H, ps, P = 300, 2, 16, 12
    slots = np.full(n, -1, np.int64)
    slots[:100] = make_slots(rng, P, ps, [0], [100])
    slots[200] = P * ps
    slots[201] = 2 ** 40
    xk, xv = values(rng, n, H, torch.bfloat16), values(rng, n, H, torch.bfloat16)
    kc_, vc_ = make_cache(rng, P, ps, H), make_cache(rng, P, ps, H)
    check_append(run_append(bsp, xk, xv, slots, kc_, vc_), xk, xv, slots, kc_, vc_)
    none = np.full(n, -1, np.int64)
    check_append(run_append(bsp, xk, xv, none, kc_, vc_), xk, xv, none, kc_, vc_)


@pytest.mark.parametrize("ps", [1, 3, 16, 40])
def test_append_with_skipped_tokens_anywhere(bsp, ps):
    """Slots of -1 between the runs of pages, single ones and long stretches, at random."""
    rng = np.random.default_rng(40 + ps)
    H, P = 2, 120
    slots, pages = [], rng.permutation(P)
    for p in pages:
        a = int(rng.integers(0, ps))
        b = int(rng.integers(a, ps)) + 1
        slots += list(range(int(p) * ps + a, int(p) * ps + b))
        slots += [-1] * int(rng.choice([0, 0, 1, 2, 15, 16, 17, 40]))
    slots = np.array(slots, np.int64)
    n = len(slots)
    xk, xv = values(rng, n, H, torch.bfloat16), values(rng, n, H, torch.bfloat16)
    kc_, vc_ = make_cache(rng, P, ps, H), make_cache(rng, P, ps, H)
    check_append(run_append(bsp, xk, xv, slots, kc_, vc_), xk, xv, slots, kc_, vc_)


def test_append_one_token_at_a_time_equals_the_oracle(bsp):
    """Twenty decode steps into the same pages, growing values: every step may raise the pages' exponents."""
    rng = np.random.default_rng(32)
    H, ps, P = 2, 8, 9
    kc_, vc_ = make_cache(rng, P, ps, H), make_cache(rng, P, ps, H)
    f8 = torch.float8_e4m3fn
    t = [dev(kc_[0]).view(f8), dev(vc_[0]).view(f8), dev(kc_[1]), dev(vc_[1])]
    pages = rng.permutation(P)
    for step in range(20):
        slots = np.array([int(pages[3 * b + step // ps]) * ps + step % ps for b in range(3)], np.int64)
        x = values(rng, 3, H, torch.bfloat16) * (1.5 ** step)
        y = values(rng, 3, H, torch.bfloat16)
        bsp.append_kv(x.cuda(), y.cuda(), dev(slots), *t)
        kc_ = kc.append(x.double().numpy(), slots, *kc_)
        vc_ = kc.append(y.double().numpy(), slots, *vc_)
    for (c, e), g8, ge in ((kc_, t[0], t[2]), (vc_, t[1], t[3])):
        assert np.array_equal(ge.cpu().numpy(), e)
        g = g8.view(torch.uint8).cpu().numpy()
        assert np.array_equal(np.where(g & 0x7f == 0x7f, 0x7f, g), np.where(c & 0x7f == 0x7f, 0x7f, c))


def test_append_slots_past_32_bits_of_bytes(bsp):
    """A pool of more than 2^32 bytes: pages at its far end are written, and only those."""
    P, ps, H = 300000, 16, 8  # 4.9 GB of codes per pool
    k8 = torch.zeros((P, ps, H, 128), dtype=torch.uint8, device="cuda")
    v8 = torch.zeros_like(k8)
    ke = torch.zeros((P, H), dtype=torch.int8, device="cuda")
    ve = torch.zeros_like(ke)
    rng = np.random.default_rng(33)
    slots = np.concatenate([np.arange((P - 1) * ps, P * ps), [5 * ps]]).astype(np.int64)
    x = values(rng, ps + 1, H, torch.bfloat16)
    f8 = torch.float8_e4m3fn
    bsp.append_kv(x.cuda(), x.cuda(), dev(slots), k8.view(f8), v8.view(f8), ke, ve)
    c0, e0 = np.zeros((2, ps, H, 128), np.uint8), np.zeros((2, H), np.int8)
    want, we = kc.append(x.double().numpy(), np.concatenate([np.arange(ps), [ps]]), c0, e0)
    for p, w in ((P - 1, 0), (5, 1)):
        assert np.array_equal(k8[p].cpu().numpy(), want[w]) and np.array_equal(v8[p].cpu().numpy(), want[w])
        assert np.array_equal(ke[p].cpu().numpy(), we[w])
    k8[P - 1], k8[5] = 0, 0
    assert not k8.any() and int((ke != 0).sum()) <= 2 * H


def test_tables_and_append_in_a_graph_on_another_stream(bsp):
    """One captured step (tables, then append through its slots, padded) replayed for three steps of growing
    requests, against the oracle."""
    rng = np.random.default_rng(34)
    B, ps, H, P, width, cap_t = 5, 4, 2, 64, 8, 24
    f8 = torch.float8_e4m3fn
    kc_, vc_ = make_cache(rng, P, ps, H), make_cache(rng, P, ps, H)
    t = [dev(kc_[0]).view(f8), dev(vc_[0]).view(f8), dev(kc_[1]), dev(vc_[1])]
    cached, new = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    free, nfree = torch.zeros(P, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    k = torch.zeros((cap_t, H, 128), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    out = bsp.PageTables.empty(B, B * width, cap_t)

    def step():
        bsp.build_page_tables(cached, new, free, nfree, table, ps, B * width, cap_t, out=out)
        bsp.append_kv(k, v, out.slot_map, *t)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()  # no new tokens: nothing is written
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    pool = rng.permutation(P).astype(np.int32)
    c = np.zeros(B, np.int32)
    bt = np.full((B, width), -1, np.int32)
    with torch.cuda.stream(s):
        for _ in range(3):
            m = rng.integers(0, 5, B).astype(np.int32)
            n = int(m.sum())
            xk, xv = values(rng, n, H, torch.bfloat16), values(rng, n, H, torch.bfloat16)
            cached.copy_(dev(c)), new.copy_(dev(m)), nfree.fill_(len(pool))
            free[:len(pool)].copy_(dev(pool))
            k[:n].copy_(xk.cuda()), v[:n].copy_(xv.cuda())
            g.replay()
            want = kc.tables(c, m, pool, len(pool), bt, ps, B * width, cap_t)
            s.synchronize()
            for f in out._fields:
                assert np.array_equal(getattr(out, f).cpu().numpy(), want[f]), f
            bt = want["block_table"]
            assert np.array_equal(table.cpu().numpy(), bt)
            kc_ = kc.append(xk.double().numpy(), want["slot_map"][:n], *kc_)
            vc_ = kc.append(xv.double().numpy(), want["slot_map"][:n], *vc_)
            pool = pool[int(want["counts"][2]):]
            c = c + m
    for (cc, e), g8, ge in ((kc_, t[0], t[2]), (vc_, t[1], t[3])):
        assert np.array_equal(ge.cpu().numpy(), e)
        gg = g8.view(torch.uint8).cpu().numpy()
        assert np.array_equal(np.where(gg & 0x7f == 0x7f, 0x7f, gg), np.where(cc & 0x7f == 0x7f, 0x7f, cc))
