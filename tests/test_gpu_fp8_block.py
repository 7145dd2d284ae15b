"""Decode and prefill over the 8-bit cache with one exponent per page and kv head,
against the fp64 oracle on the values that the codes stand for.

Bounds, from the arithmetic (u = half a step of the type that a token's weight is
rounded to before the product with V: 2^-11 for f16 in decode, 2^-8 for bf16 in
prefill; A = sum_j p_j |v_j|, from the oracle):
- a score is an fp32 sum of 128 products, truncated at most 2^-23 of the running sum
  in each of up to 32 additions, and a few more roundings: |ds| <= 2^-18 (1 +
  scale * |q| |k|), and with a soft-cap c its tanh's 2^-21 c on top; LSE moves by no
  more than the largest ds (plus its own logarithm, within the same 2^-18);
- O: every weight by a factor 1 +- (u + 2 ds), the weights under f16's normal range
  by 2^-25 of the largest (at most 448 / |code| of it in a dimension: taken as 2^-25
  n_keys against the row's largest A, times 448), and half a bf16 step of O itself.
"""
import ctypes
import math

import numpy as np
import pytest
import torch

import oracle
import workloads
from gpu_helpers import half_ulp_bf16, lib
from oracle import kv_cache as kc

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bsp():
    return lib()


def cache8(b, seed, ke=(-8, -5), ve=(-8, -4)):
    """Codes and exponents of a batch: its normal values as codes (NaN poison as the NaN code), exponents drawn per
    page and head, and 127 in pages that nobody uses."""
    rng = np.random.default_rng(seed)
    out = []
    used = np.zeros(b.k_pages.shape[0], bool)
    used[b.kv_indices] = True
    for x, (lo, hi) in ((b.k_pages, ke), (b.v_pages, ve)):
        codes = (x.float() * 60).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
        e = rng.integers(lo, hi, (x.shape[0], x.shape[2]), endpoint=True)
        e[~used] = 127
        out += [codes, e.astype(np.int8)]
    return out


def run_block(bsp, b, c8, num_ctas=None, sink=None, stream=None, repeats=1, **kw):
    decode = not b.causal and b.is_decode
    pa = bsp.PagedAttention("decode" if decode else "prefill", b.num_qo_heads, b.num_kv_heads, 128, b.page_size,
                            b.causal, torch.bfloat16, max_batch=b.batch, max_qo_tokens=max(1, int(b.qo_indptr[-1])),
                            num_ctas=num_ctas, window_left=b.window_left, logits_soft_cap=b.soft_cap, **kw)
    pa.plan(b.kv_indptr, b.last_page_len, qo_indptr=None if decode else b.qo_indptr)
    k8, ke, v8, ve = (torch.from_numpy(a).cuda() for a in c8)
    f8 = torch.float8_e4m3fn
    idx = torch.from_numpy(np.ascontiguousarray(b.kv_indices, np.int32)).cuda()
    sk = None if sink is None else torch.tensor(sink, dtype=torch.float32, device="cuda")
    q = b.q.cuda()
    torch.cuda.synchronize()
    for _ in range(repeats):
        out, lse = pa.run(q, k8.view(f8), v8.view(f8), idx, b.sm_scale, k_exp=ke, v_exp=ve, sink=sk, stream=stream)
    torch.cuda.synchronize()
    return out, lse, pa


def reference(b, c8, sink=None):
    k, v = kc.values(c8[0], c8[1]), kc.values(c8[2], c8[3])
    O, L = oracle.attention_of(b, k=k, v=v, sink=sink)
    A, _ = oracle.attention_of(b, k=k, v=np.abs(v), sink=sink)
    used = np.unique(b.kv_indices)
    kn = np.nan_to_num(k[used])
    qk = b.sm_scale * np.sqrt((b.q.float().numpy() ** 2).sum(-1)).max(initial=0) * \
        np.sqrt((kn ** 2).sum(-1)).max(initial=0)
    return O, L, A, qk


def check(out, lse, ref, u, b):
    O, L, A, qk = ref
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    empty = np.isneginf(L)
    assert np.array_equal(np.isneginf(l), empty) and np.all(o[empty] == 0) and np.isfinite(o).all()
    ds = 2.0 ** -18 * (1 + qk) + 2.0 ** -21 * b.soft_cap
    n = int(b.kv_lens.max(initial=0))
    bound = half_ulp_bf16(O) * (1 + 2.0 ** -6) + (u + 2 * ds) * A * (1 + 2.0 ** -7)
    if u < 2.0 ** -10:
        bound = bound + 448 * n * 2.0 ** -25 * A.max(-1, keepdims=True)
    excess = (np.abs(o - O) - bound).max(initial=0)
    assert excess <= 0, f"O beyond its bound by {excess}"
    fin = ~empty
    dl = np.abs(l[fin] - L[fin]).max(initial=0)
    assert dl <= 2 * ds, f"LSE off by {dl}, bound {2 * ds}"


DECODE = [
    # (seed, kv lens, H_qo, H_kv, page, num_ctas, window, cap)
    (201, [3000, 17, 900, 4100, 1, 250, 64, 65], 32, 8, 16, 29, -1, 0.0),   # splits, ragged tails
    (202, [5000, 33, 129], 32, 8, 8, 17, -1, 0.0),                          # one exponent per 8 tokens
    (203, [2048, 1000, 7], 12, 4, 32, 11, -1, 0.0),                         # g = 3
    (204, [4000, 300], 64, 8, 64, 9, -1, 0.0),                              # g = 8
    (205, [6000, 130, 2], 32, 2, 128, 23, -1, 0.0),                         # g = 16, two boxes per page
    (206, [3000, 900, 4100], 32, 8, 16, 13, 700, 1.5),                      # window and soft-cap
    (207, [0, 40, 0, 1], 32, 8, 16, 5, -1, 0.0),                            # empty requests
    (208, [700, 1, 3000, 256, 257], 32, 8, 1, 19, -1, 0.0),                 # page size 1: an exponent per token
    (209, [1000, 4, 333], 9, 1, 5, 7, -1, 0.0),                             # odd pages, g = 9, one kv head
    (210, [129, 2000], 8, 8, 12, None, 300, 30.0),                          # g = 1
    (211, [1500, 3], 32, 2, 4, 6, -1, 0.0),                                 # g = 16 through the gather
    (212, [1], 5, 1, 16, None, -1, 0.0),                                    # one token
    (213, [2500, 70], 40, 8, 100, 8, -1, 0.0),                              # page not a power of two
]


@pytest.mark.parametrize("case", DECODE, ids=[f"d{c[0]}" for c in DECODE])
def test_decode(bsp, case):
    seed, kv, hq, hk, ps, C, w, cap = case
    b = workloads.paged_batch(seed, [1] * len(kv), kv, hq, hk, 128, ps, "bf16", extra_pages=3)
    b.window_left, b.soft_cap = w, cap
    c8 = cache8(b, seed)
    out, lse, pa = run_block(bsp, b, c8, num_ctas=C, repeats=2)
    check(out, lse, reference(b, c8), 2.0 ** -11, b)
    assert pa.check_device_error() == 0


@pytest.mark.parametrize("case", DECODE, ids=[f"d{c[0]}" for c in DECODE])
def test_decode_with_exponents_gathered_first(bsp, case):
    """The C entry without a region, with one, with a larger one, and with one that the table outgrew since the
    capture: the same bits."""
    seed, kv, hq, hk, ps, C, w, cap = case
    b = workloads.paged_batch(seed, [1] * len(kv), kv, hq, hk, 128, ps, "bf16", extra_pages=3)
    b.window_left, b.soft_cap = w, cap
    few = workloads.paged_batch(seed, [1] * len(kv), [min(n, 1 + i) for i, n in enumerate(kv)], hq, hk, 128, ps, "bf16")
    c8 = cache8(b, seed)
    pa = bsp.PagedAttention("decode", hq, hk, 128, ps, False, torch.bfloat16, max_batch=b.batch, max_qo_tokens=b.batch,
                            num_ctas=C, window_left=w, logits_soft_cap=cap)
    k8, ke, v8, ve = (torch.from_numpy(a).cuda() for a in c8)
    idx = torch.from_numpy(np.ascontiguousarray(b.kv_indices, np.int32)).cuda()
    q = b.q.cuda()
    n, got = -(-len(idx) // 16) * 16, []
    for entries in (0, n, n + 32, None):
        region = torch.full(((n if entries is None else entries) * 2 * hk,), 0x7f, dtype=torch.uint8, device="cuda")
        o, l = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")

        def run(nbytes):
            rc = pa.lib.bsp_decode_run_fp8_block(
                ctypes.byref(pa.info), q.data_ptr(), k8.data_ptr(), v8.data_ptr(), ke.data_ptr(), ve.data_ptr(),
                idx.data_ptr(), k8.shape[0], b.sm_scale, o.data_ptr(), l.data_ptr(), region.data_ptr() if nbytes else None,
                nbytes, pa.workspace.data_ptr(), torch.cuda.current_stream().cuda_stream)
            assert rc == 0
        if entries is None:
            pa.plan(few.kv_indptr, few.last_page_len, qo_indptr=few.qo_indptr)
            small = -(-pa.info.num_table_pages // 16) * 16 * 2 * hk
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                run(small)
            pa.plan(b.kv_indptr, b.last_page_len, qo_indptr=b.qo_indptr)
            g.replay()
            torch.cuda.synchronize()
            assert (region[small:] == 0x7f).all()
        else:
            pa.plan(b.kv_indptr, b.last_page_len, qo_indptr=b.qo_indptr)
            run(region.numel())
            torch.cuda.synchronize()
        assert pa.check_device_error() == 0
        got.append((o, l))
    check(*got[0], reference(b, c8), 2.0 ** -11, b)
    for o, l in got[1:]:
        assert torch.equal(o, got[0][0]) and torch.equal(l, got[0][1])


def test_decode_gathers_by_the_rule(bsp):
    """Pages of one token and work enough: run() gathers; a page id outside the pool reads as zeros all the same."""
    b = workloads.paged_batch(248, [1] * 3, [9000, 4100, 300], 8, 2, 128, 1, "bf16", extra_pages=3)
    c8 = cache8(b, 248)
    b.kv_indices[5] = b.kv_indices[9001] = -1
    pa = bsp.PagedAttention("decode", 8, 2, 128, 1, False, torch.bfloat16, max_batch=3, max_qo_tokens=3, num_ctas=4)
    pa.plan(b.kv_indptr, b.last_page_len, qo_indptr=b.qo_indptr)
    assert pa.lib.bsp_decode_fp8_region_size(ctypes.byref(pa.info)) == 13408 * 2 * 2
    k8, ke, v8, ve = (torch.from_numpy(a).cuda() for a in c8)
    f8 = torch.float8_e4m3fn
    idx = torch.from_numpy(np.ascontiguousarray(b.kv_indices, np.int32)).cuda()
    o, l = pa.run(b.q.cuda(), k8.view(f8), v8.view(f8), idx, k_exp=ke, v_exp=ve)
    torch.cuda.synchronize()
    assert pa.check_device_error() == 0x302
    zero = [np.concatenate([c, np.zeros_like(c[:1])]) for c in c8]
    b.kv_indices[[5, 9001]] = len(c8[0])
    check(o, l, reference(b, zero), 2.0 ** -11, b)


PREFILL = [
    # (seed, qo lens, kv lens, H_qo, H_kv, page, num_ctas, window, cap)
    (221, [100, 37, 1, 300], [100, 300, 5, 300], 32, 8, 16, None, -1, 0.0),
    (222, [33, 260], [1033, 700], 8, 8, 1, 13, -1, 0.0),                    # page size 1, g = 1
    (223, [70, 0, 5], [2000, 40, 5], 32, 2, 64, 17, -1, 0.0),               # splits, an empty request, g = 16
    (224, [129, 128], [129, 1000], 16, 4, 12, 9, 200, 30.0),                # window and soft-cap, odd pages
    (225, [513], [4000], 8, 1, 128, 21, -1, 0.0),                           # chunk behind a long cache
    (226, [6, 2], [3, 2], 16, 2, 8, 4, -1, 0.0),                            # rows that see no key
    (227, [1, 1], [700, 1], 4, 1, 5, None, -1, 0.0),
    # many short items per CTA: none, one, two or four tiles each, ends on and off a tile
    (228, [1 + 7 * i % 50 for i in range(40)], [(37 * i) % 400 if i % 5 else 128 * (i % 4) for i in range(40)], 16, 2, 8, 3,
     -1, 0.0),
    (229, [1 + 11 * i % 90 for i in range(24)], [(53 * i) % 700 for i in range(24)], 8, 2, 32, 2, 100, 0.0),
    (230, [1 + 7 * i % 50 for i in range(24)], [(37 * i) % 400 for i in range(24)], 16, 2, 6, 3, -1, 0.0),
]


@pytest.mark.parametrize("case", PREFILL, ids=[f"p{c[0]}" for c in PREFILL])
def test_prefill(bsp, case):
    seed, qo, kv, hq, hk, ps, C, w, cap = case
    b = workloads.paged_batch(seed, qo, kv, hq, hk, 128, ps, "bf16", causal=True, extra_pages=2)
    b.window_left, b.soft_cap = w, cap
    c8 = cache8(b, seed)
    out, lse, pa = run_block(bsp, b, c8, num_ctas=C, repeats=2)
    check(out, lse, reference(b, c8), 2.0 ** -8, b)
    assert pa.check_device_error() == 0


@pytest.mark.parametrize("case", PREFILL, ids=[f"p{c[0]}" for c in PREFILL])
def test_prefill_converted_before_and_inside_the_kernel(bsp, case):
    """The C entry with a region (larger than needed, full of NaN) and without one: the same tiles, the same bits."""
    seed, qo, kv, hq, hk, ps, C, w, cap = case
    b = workloads.paged_batch(seed, qo, kv, hq, hk, 128, ps, "bf16", causal=True, extra_pages=2)
    b.window_left, b.soft_cap = w, cap
    c8 = cache8(b, seed, ke=(-20, -5), ve=(-12, 3))
    pa = bsp.PagedAttention("prefill", hq, hk, 128, ps, True, torch.bfloat16, max_batch=b.batch,
                            max_qo_tokens=int(b.qo_indptr[-1]), num_ctas=C, window_left=w, logits_soft_cap=cap)
    pa.plan(b.kv_indptr, b.last_page_len, qo_indptr=b.qo_indptr)
    k8, ke, v8, ve = (torch.from_numpy(a).cuda() for a in c8)
    idx = torch.from_numpy(np.ascontiguousarray(b.kv_indices, np.int32)).cuda()
    q = b.q.cuda()
    got = []
    for pages in (0, len(b.kv_indices), len(b.kv_indices) + 7):
        region = torch.full((pages * ps * hk * 256,), float("nan"), dtype=torch.bfloat16, device="cuda")
        o, l = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
        rc = pa.lib.bsp_prefill_run_fp8_block(
            ctypes.byref(pa.info), q.data_ptr(), k8.data_ptr(), v8.data_ptr(), ke.data_ptr(), ve.data_ptr(), idx.data_ptr(),
            k8.shape[0], b.sm_scale, o.data_ptr(), l.data_ptr(), region.data_ptr() if pages else None, region.numel() * 2,
            pa.workspace.data_ptr(), torch.cuda.current_stream().cuda_stream)
        assert rc == 0
        torch.cuda.synchronize()
        assert pa.check_device_error() == 0
        got.append((o, l))
    check(*got[0], reference(b, c8), 2.0 ** -8, b)
    for o, l in got[1:]:
        assert torch.equal(o, got[0][0]) and torch.equal(l, got[0][1])


def test_region_too_small_for_a_later_plan(bsp):
    """A captured run whose region holds the captured plan's pages, replayed after a plan with more: the status word."""
    a = workloads.paged_batch(240, [300], [300], 8, 2, 128, 16, "bf16", causal=True)
    b = workloads.paged_batch(241, [300], [900], 8, 2, 128, 16, "bf16", causal=True)
    pa = bsp.PagedAttention("prefill", 8, 2, 128, 16, True, torch.bfloat16, max_batch=1, max_qo_tokens=300, num_ctas=4)
    k8, ke, v8, ve = (torch.from_numpy(x).cuda() for x in cache8(b, 241))
    f8 = torch.float8_e4m3fn
    idx = torch.arange(60, dtype=torch.int32, device="cuda")
    q = a.q.cuda()
    o, l = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")

    def run():
        pa.run(q, k8.view(f8), v8.view(f8), idx, out=o, lse=l, k_exp=ke, v_exp=ve)
    pa.plan(a.kv_indptr, a.last_page_len, qo_indptr=a.qo_indptr)
    assert pa.lib.bsp_prefill_fp8_region_size(ctypes.byref(pa.info)) > 0
    run()
    torch.cuda.synchronize()
    want = o.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    g.replay()
    assert pa.check_device_error() == 0 and torch.equal(o, want)
    pa.plan(b.kv_indptr, b.last_page_len, qo_indptr=b.qo_indptr)
    g.replay()
    assert pa.check_device_error() == 0x303
    pa.plan(a.kv_indptr, a.last_page_len, qo_indptr=a.qo_indptr)
    g.replay()
    assert pa.check_device_error() == 0 and torch.equal(o, want)


@pytest.mark.parametrize("kind", ["decode", "prefill"])
@pytest.mark.parametrize("ps", [1, 16])
def test_exponents_far_apart(bsp, kind, ps):
    """V exponents over 120 binades and K exponents over 20: small blocks that the softmax prefers stay exact beside
    huge ones that it does not."""
    qo = [1, 1] if kind == "decode" else [40, 9]
    b = workloads.paged_batch(231, qo, [900, 77], 16, 2, 128, ps, "bf16", causal=kind == "prefill", extra_pages=1)
    c8 = cache8(b, 231, ke=(-25, -5), ve=(-70, 50))
    out, lse, _ = run_block(bsp, b, c8, num_ctas=7)
    check(out, lse, reference(b, c8), 2.0 ** -11 if kind == "decode" else 2.0 ** -8, b)


@pytest.mark.parametrize("kind", ["decode", "prefill"])
def test_a_dominant_small_block(bsp, kind):
    """One block holds the key that the queries want and tiny values; all others hold values 2^40 times larger at
    scores that leave them 2^-60: the answer is the tiny block's."""
    qo = [1] if kind == "decode" else [3]
    b = workloads.paged_batch(232, qo, [320], 8, 1, 128, 16, "bf16", causal=kind == "prefill")
    b.q = torch.ones_like(b.q)
    k8, ke, v8, ve = cache8(b, 232, ke=(0, 0), ve=(0, 0))
    k8[:] = 0xb8  # -1
    page = int(b.kv_indices[4])
    k8[page] = 0x38  # 1
    ke[:] = 1        # scores -+ 2 * 128 / sqrt(128): 45 apart, 2^-65
    ve[:], ve[page] = 20, -20
    c8 = [k8, ke, v8, ve]
    out, lse, _ = run_block(bsp, b, c8, num_ctas=3)
    check(out, lse, reference(b, c8), 2.0 ** -11 if kind == "decode" else 2.0 ** -8, b)


@pytest.mark.parametrize("kind", ["decode", "prefill"])
def test_sink_and_empty(bsp, kind):
    qo = [1, 1, 1] if kind == "decode" else [40, 3, 2]
    b = workloads.paged_batch(233, qo, [3000, 0, 70], 32, 8, 128, 16, "bf16", causal=kind == "prefill", extra_pages=1)
    c8 = cache8(b, 233)
    sk = np.random.default_rng(233).uniform(-2.0, 4.0, size=32)
    out, lse, _ = run_block(bsp, b, c8, num_ctas=19, sink=sk)
    check(out, lse, reference(b, c8, sink=sk.astype(np.float32)), 2.0 ** -11 if kind == "decode" else 2.0 ** -8, b)


def test_non_causal_prefill_and_another_stream(bsp):
    b = workloads.paged_batch(234, [50, 20], [300, 77], 16, 4, 128, 16, "bf16")
    c8 = cache8(b, 234)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        out, lse, _ = run_block(bsp, b, c8, num_ctas=5)
    check(out, lse, reference(b, c8), 2.0 ** -8, b)


def test_nan_codes_of_valid_tokens_reach_their_request_alone(bsp):
    for causal, qo in ((False, [1, 1]), (True, [20, 30])):
        b = workloads.paged_batch(235, qo, [200, 300], 8, 2, 128, 16, "bf16", causal=causal)
        c8 = cache8(b, 235)
        c8[2][b.kv_indices[2], 3, 1, 7] = 0x7f  # V, request 0, kv head 1, dimension 7
        out, _, _ = run_block(bsp, b, c8, num_ctas=1)
        o = out.float().cpu().numpy()
        last = qo[0] - 1
        assert np.isnan(o[last, 4:, 7]).all() and np.isfinite(o[last, :4]).all() and np.isfinite(o[qo[0]:]).all()


def test_long_cache_past_32_bits(bsp):
    """A pool whose codes pass 2^32 bytes and whose rows pass int32 elements: the far pages, decode and prefill."""
    P, ps, H = 300000, 16, 8
    b = workloads.paged_batch(236, [1, 1], [40, 300], 32, 8, 128, ps, "bf16")
    c8 = cache8(b, 236)
    n = c8[0].shape[0]
    f8 = torch.float8_e4m3fn
    k8 = torch.full((P, ps, H, 128), 0x7f, dtype=torch.uint8, device="cuda")
    v8 = torch.full_like(k8, 0x7f)
    ke = torch.full((P, H), 100, dtype=torch.int8, device="cuda")
    ve = torch.full_like(ke, 100)
    for t, a in zip((k8, ke, v8, ve), c8):
        t[P - n:] = torch.from_numpy(a).cuda()
    idx = torch.from_numpy(np.ascontiguousarray(b.kv_indices, np.int32)).cuda() + (P - n)
    for mode in ("decode", "prefill"):
        pa = bsp.PagedAttention(mode, 32, 8, 128, ps, False, torch.bfloat16, max_batch=2, max_qo_tokens=2)
        pa.plan(b.kv_indptr, b.last_page_len, qo_indptr=None if mode == "decode" else b.qo_indptr)
        out, lse = pa.run(b.q.cuda(), k8.view(f8), v8.view(f8), idx, b.sm_scale, k_exp=ke, v_exp=ve)
        torch.cuda.synchronize()
        check(out, lse, reference(b, c8), 2.0 ** -11 if mode == "decode" else 2.0 ** -8, b)


@pytest.mark.parametrize("mode", ["decode", "prefill"])
def test_full_size(bsp, mode):
    """64 requests of up to 8192 tokens (decode); 16 ragged prompts (prefill, a stratified part of the rows)."""
    if mode == "decode":
        b = workloads.batched_decode_bf16()
    else:
        b = workloads.paged_batch(237, [1500, 700, 64, 2048], [1500, 2700, 64, 2048], 32, 8, 128, 16, "bf16",
                                  causal=True)
    c8 = cache8(b, 237)
    out, lse, pa = run_block(bsp, b, c8, repeats=2)
    check(out, lse, reference(b, c8), 2.0 ** -11 if mode == "decode" else 2.0 ** -8, b)
    assert pa.check_device_error() == 0


def test_serving_loop(bsp):
    """Prompts, then decode steps: tables, append, plan and attention as a server runs them, the decode step captured
    once and replayed, every output against the oracle on the oracle's own cache."""
    rng = np.random.default_rng(238)
    B, ps, hq, hk, P, width = 4, 16, 16, 4, 80, 16
    f8, i32 = torch.float8_e4m3fn, torch.int32
    codes = [np.full((P, ps, hk, 128), 0x7f, np.uint8) for _ in range(2)]
    exps = [np.full((P, hk), 90, np.int8) for _ in range(2)]
    k8, v8 = (torch.from_numpy(c).cuda().view(f8) for c in codes)
    ke, ve = (torch.from_numpy(e).cuda() for e in exps)
    bt = np.full((B, width), -1, np.int32)
    table = torch.from_numpy(bt).cuda()
    pool = rng.permutation(P).astype(np.int32)
    free = torch.zeros(P, dtype=i32, device="cuda")
    nfree, lens_d, new_d = (torch.zeros(n, dtype=i32, device="cuda") for n in (1, B, B))
    cached = np.zeros(B, np.int64)

    def values(n, h):
        return torch.from_numpy(rng.standard_normal((n, h, 128)) * np.exp2(rng.uniform(-2, 2, (n, 1, 1)))).bfloat16()

    def load(m):
        lens_d.copy_(torch.from_numpy(cached.astype(np.int32)))
        new_d.copy_(torch.from_numpy(m.astype(np.int32)))
        free[:len(pool)].copy_(torch.from_numpy(pool))
        nfree.fill_(len(pool))

    def expect(m, q, xk, xv, causal):
        nonlocal codes, exps, bt, pool
        t = kc.tables(cached, m, pool, len(pool), bt, ps, B * width, len(q))
        bt, pool = t["block_table"], pool[int(t["counts"][2]):]
        for j, x in enumerate((xk, xv)):
            codes[j], exps[j] = kc.append(x.double().numpy(), t["slot_map"], codes[j], exps[j])
        n_pages = int(t["counts"][0])
        wb = workloads.PagedBatch("step", "bf16", hq, hk, 128, ps, causal, 1 / math.sqrt(128), t["qo_indptr"],
                                  t["kv_indptr"], t["kv_indices"][:n_pages], t["last_page_len"], q, torch.zeros(1),
                                  torch.zeros(1))
        return t, wb, reference(wb, [codes[0], exps[0], codes[1], exps[1]])

    # prompts
    m = np.array([70, 1, 33, 16])
    n = int(m.sum())
    q, xk, xv = values(n, hq), values(n, hk), values(n, hk)
    load(m)
    t = bsp.build_page_tables(lens_d, new_d, free, nfree, table, ps, B * width, n)
    bsp.append_kv(xk.cuda(), xv.cuda(), t.slot_map, k8, v8, ke, ve)
    pp = bsp.PagedAttention("prefill", hq, hk, 128, ps, True, torch.bfloat16, max_batch=B, max_qo_tokens=n)
    want, wb, ref = expect(m, q, xk, xv, True)
    pp.plan(want["kv_indptr"], want["last_page_len"], qo_indptr=want["qo_indptr"])
    out, lse = pp.run(q.cuda(), k8, v8, t.kv_indices, k_exp=ke, v_exp=ve)
    torch.cuda.synchronize()
    check(out, lse, ref, 2.0 ** -8, wb)
    cached += m
    # decode steps
    ones = np.ones(B, np.int64)
    qd = torch.zeros((B, hq, 128), dtype=torch.bfloat16, device="cuda")
    kd, vd = (torch.zeros((B, hk, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    o, l = torch.empty_like(qd), torch.empty((B, hq), device="cuda")
    tabs = bsp.PageTables.empty(B, B * width, B)
    pa = bsp.PagedAttention("decode", hq, hk, 128, ps, False, torch.bfloat16, max_batch=B)

    def step():
        bsp.build_page_tables(lens_d, new_d, free, nfree, table, ps, B * width, B, out=tabs)
        bsp.append_kv(kd, vd, tabs.slot_map, k8, v8, ke, ve)
        pa.run(qd, k8, v8, tabs.kv_indices, out=o, lse=l, k_exp=ke, v_exp=ve)
    g = None
    for i in range(20):
        q, xk, xv = values(B, hq), values(B, hk), values(B, hk)
        want, wb, ref = expect(ones, q, xk, xv, False)
        grown = want["kv_indptr"]
        load_pool = np.concatenate([want["block_table"][b, -(-int(cached[b]) // ps):-(-int(cached[b] + 1) // ps)]
                                    for b in range(B)] + [pool]).astype(np.int32)
        lens_d.copy_(torch.from_numpy(cached.astype(np.int32)))
        new_d.fill_(1)
        free[:len(load_pool)].copy_(torch.from_numpy(load_pool))
        nfree.fill_(len(load_pool))
        qd.copy_(q), kd.copy_(xk), vd.copy_(xv)
        pa.plan(grown, want["last_page_len"])
        if i == 0:
            step()
        else:
            if g is None:
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g):
                    step()
            g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(tabs.slot_map.cpu().numpy(), want["slot_map"])
        assert np.array_equal(table.cpu().numpy(), bt)
        check(o, l, ref, 2.0 ** -11, wb)
        cached += 1
    assert pa.check_device_error() == 0


@pytest.mark.parametrize("kind", ["decode", "prefill"])
@pytest.mark.parametrize("ps", [3, 16])
def test_page_ids_outside_the_pool_read_as_zeros(bsp, kind, ps):
    """An id past the pool and a negative one: zero keys and values, the status word, the other rows untouched."""
    qo = [1, 1] if kind == "decode" else [9, 12]
    b = workloads.paged_batch(239, qo, [200, 90], 8, 2, 128, ps, "bf16", causal=kind == "prefill")
    c8 = cache8(b, 239)
    z = [np.concatenate([a, np.zeros((1,) + a.shape[1:], a.dtype)]) for a in c8]
    b.kv_indices = b.kv_indices.copy()
    P = c8[0].shape[0]
    at = [0, 2]
    b.kv_indices[at] = P
    ref = reference(b, z)
    b.kv_indices[at[0]], b.kv_indices[at[1]] = P + 5, -1
    out, lse, pa = run_block(bsp, b, c8, num_ctas=4)
    check(out, lse, ref, 2.0 ** -11 if kind == "decode" else 2.0 ** -8, b)
    assert pa.check_device_error() == 0x302 and pa.check_device_error() == 0


def test_streams_given_to_the_calls(bsp):
    """Every call on a stream passed to it, another one current, the copy region included."""
    b = workloads.paged_batch(242, [300, 64], [300, 200], 8, 2, 128, 16, "bf16", causal=True)
    c8 = cache8(b, 242)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, lse, pa = run_block(bsp, b, c8, num_ctas=3, stream=s)
    assert pa.lib.bsp_prefill_fp8_region_size(ctypes.byref(pa.info)) > 0
    check(out, lse, reference(b, c8), 2.0 ** -8, b)
    d = workloads.paged_batch(243, [1, 1], [300, 200], 8, 2, 128, 16, "bf16")
    d8 = cache8(d, 243)
    out, lse, _ = run_block(bsp, d, d8, num_ctas=3, stream=s)
    check(out, lse, reference(d, d8), 2.0 ** -11, d)


def test_run_refuses(bsp):
    """Shapes, types and sizes that do not go with the plan or the pools."""
    b = workloads.paged_batch(244, [1, 1], [40, 20], 8, 2, 128, 16, "bf16")
    k8, ke, v8, ve = (torch.from_numpy(a).cuda() for a in cache8(b, 244))
    f8 = torch.float8_e4m3fn
    k8, v8, q = k8.view(f8), v8.view(f8), b.q.cuda()
    idx = torch.from_numpy(np.ascontiguousarray(b.kv_indices, np.int32)).cuda()
    pa = bsp.PagedAttention("decode", 8, 2, 128, 16, False, torch.bfloat16, max_batch=2)
    with pytest.raises(RuntimeError):
        pa.run(q, k8, v8, idx, k_exp=ke, v_exp=ve)  # no plan
    pa.plan(b.kv_indptr, b.last_page_len)
    ok = dict(q=q, k_pages=k8, v_pages=v8, kv_indices=idx, k_exp=ke, v_exp=ve)
    for bad in (dict(k_exp=None), dict(v_exp=None), dict(k_scale=2.0), dict(q=q[:1]), dict(q=q[:, :4]), dict(q=q.float()),
                dict(k_pages=k8.view(torch.uint8)), dict(k_pages=k8[:, :8]), dict(v_pages=v8[:1]), dict(k_exp=ke[:1]),
                dict(k_exp=ke.short()), dict(kv_indices=idx[:1]), dict(kv_indices=idx.long()), dict(out=q[:1].clone()),
                dict(out=q.float()), dict(lse=torch.zeros(2, 4, device="cuda")), dict(q=q.cpu())):
        with pytest.raises(ValueError):
            pa.run(**{**ok, **bad})
    g17 = bsp.PagedAttention("decode", 34, 2, 128, 16, False, torch.bfloat16, max_batch=2)
    g17.plan(b.kv_indptr, b.last_page_len)
    with pytest.raises(bsp.BspError, match="UNSUPPORTED"):
        g17.run(torch.zeros(2, 34, 128, dtype=torch.bfloat16, device="cuda"), k8, v8, idx, k_exp=ke, v_exp=ve)
    f32 = bsp.PagedAttention("decode", 8, 2, 128, 16, False, torch.float32, max_batch=2)
    f32.plan(b.kv_indptr, b.last_page_len)
    with pytest.raises(ValueError):
        f32.run(**ok)


def test_prefill_in_the_workspace_region(bsp):
    """max_gather_pages: the copy goes into the plan's workspace, nothing is allocated by the run, the captured run
    follows a plan with a larger table within the bound."""
    a = workloads.paged_batch(245, [300], [300], 8, 2, 128, 16, "bf16", causal=True)
    b = workloads.paged_batch(246, [300], [900], 8, 2, 128, 16, "bf16", causal=True)
    pa = bsp.PagedAttention("prefill", 8, 2, 128, 16, True, torch.bfloat16, max_batch=1, max_qo_tokens=300, num_ctas=4,
                            max_gather_pages=57)
    f8 = torch.float8_e4m3fn
    P = b.k_pages.shape[0]
    pool = [torch.zeros((P,) + x.shape[1:], dtype=torch.from_numpy(x).dtype, device="cuda") for x in cache8(b, 246)]
    idx = torch.zeros(64, dtype=torch.int32, device="cuda")
    q, o, l = a.q.cuda(), torch.empty_like(a.q, device="cuda"), torch.empty(a.q.shape[:2], device="cuda")

    def load(x, c8):
        for t, h in zip(pool, c8):
            t[:h.shape[0]].copy_(torch.from_numpy(h))
        idx[:len(x.kv_indices)].copy_(torch.from_numpy(np.ascontiguousarray(x.kv_indices, np.int32)))
        q.copy_(x.q)
        pa.plan(x.kv_indptr, x.last_page_len, qo_indptr=x.qo_indptr)

    def run():
        pa.run(q, pool[0].view(f8), pool[2].view(f8), idx, out=o, lse=l, k_exp=pool[1], v_exp=pool[3])
    ca, cb = cache8(a, 245), cache8(b, 246)
    load(a, ca)
    run()
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    run()
    assert torch.cuda.max_memory_allocated() == before
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for x, c in ((a, ca), (b, cb)):
        load(x, c)
        o.fill_(9.0)
        g.replay()
        torch.cuda.synchronize()
        check(o, l, reference(x, c), 2.0 ** -8, x)
    assert pa.check_device_error() == 0


@pytest.mark.parametrize("mode", ["decode", "prefill"])
def test_no_requests_and_no_keys(bsp, mode):
    """An empty batch, and a batch whose requests are all empty: O = 0, LSE = -inf."""
    b = workloads.paged_batch(247, [1, 1], [40, 20], 8, 2, 128, 16, "bf16")
    k8, ke, v8, ve = (torch.from_numpy(a).cuda() for a in cache8(b, 247))
    f8 = torch.float8_e4m3fn
    pa = bsp.PagedAttention(mode, 8, 2, 128, 16, False, torch.bfloat16, max_batch=4, max_qo_tokens=8)
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    pa.plan([0], [], qo_indptr=[0])
    o, l = pa.run(torch.zeros(0, 8, 128, dtype=torch.bfloat16, device="cuda"), k8.view(f8), v8.view(f8), none, k_exp=ke,
                  v_exp=ve)
    assert o.shape == (0, 8, 128) and l.shape == (0, 8)
    pa.plan([0, 0, 0], [0, 0], qo_indptr=[0, 1, 2])
    o, l = pa.run(b.q.cuda(), k8.view(f8), v8.view(f8), none, k_exp=ke, v_exp=ve)
    torch.cuda.synchronize()
    assert (o == 0).all() and torch.isneginf(l).all() and pa.check_device_error() == 0


@pytest.mark.parametrize("mode", ["decode", "prefill"])
def test_runs_of_one_object_after_each_other(bsp, mode):
    """A sink in one run only, a refused run in between, and a plan that needs more pages than the tensors before."""
    a = workloads.paged_batch(249, [1, 1], [40, 20], 8, 2, 128, 16, "bf16")
    b = workloads.paged_batch(250, [1, 1], [400, 90], 8, 2, 128, 16, "bf16")
    f8, sink = torch.float8_e4m3fn, np.linspace(-1, 4, 8)
    pa = bsp.PagedAttention(mode, 8, 2, 128, 16, False, torch.bfloat16, max_batch=2, max_qo_tokens=2)
    t = {}
    for x in (a, b):
        c8 = cache8(x, 249)
        k8, ke, v8, ve = (torch.from_numpy(z).cuda() for z in c8)
        idx = torch.from_numpy(np.ascontiguousarray(x.kv_indices, np.int32)).cuda()
        t[x.batch, int(x.kv_lens[0])] = (x.q.cuda(), k8.view(f8), v8.view(f8), idx, ke, ve)
        q, k, v, idx, ke, ve = t[x.batch, int(x.kv_lens[0])]
        pa.plan(x.kv_indptr, x.last_page_len, qo_indptr=x.qo_indptr)
        if x is b:  # the tensors of the plan before
            o = t[2, 40]
            with pytest.raises(ValueError, match="kv_indices"):
                pa.run(*o[:4], k_exp=o[4], v_exp=o[5])
        u = 2.0 ** -11 if mode == "decode" else 2.0 ** -8
        s = torch.tensor(sink, dtype=torch.float32, device="cuda")
        for use in (False, True, False):
            o, l = pa.run(q, k, v, idx, k_exp=ke, v_exp=ve, sink=s if use else None)
            torch.cuda.synchronize()
            check(o, l, reference(x, c8, sink if use else None), u, x)
            with pytest.raises(ValueError, match="k_exp"):
                pa.run(q, k, v, idx, k_exp=ke[:1], v_exp=ve)
    assert pa.check_device_error() == 0
