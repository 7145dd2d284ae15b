"""Attention over the 8-bit cache where weights, queries and masked values are far from ordinary; decode against the fp64
oracle within the row-wise bounds of fp8_bounds.py."""
import numpy as np
import pytest
import torch

import oracle
import workloads
from fp8_bounds import check, decode_bounds
from gpu_helpers import lib
from oracle import fp8
from oracle import kv_cache as kc
from test_gpu_fp8_block import DECODE, cache8, run_block

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bsp():
    return lib()


def check_decode(bsp, b, c8, **kw):
    """One run against the oracle; returns its outputs."""
    out, lse, pa = run_block(bsp, b, c8, **kw)
    k, v = kc.values(c8[0], c8[1]), kc.values(c8[2], c8[3])
    O, L = oracle.attention_of(b, k=k, v=v)
    A, _ = oracle.attention_of(b, k=k, v=np.abs(v))
    check(out.double().cpu().numpy(), lse.double().cpu().numpy(), O, L,
          *decode_bounds(b, k, fp8.dequantize(c8[2], 1.0), c8[3], O, L, A))
    assert pa.check_device_error() == 0
    return out, lse


# ---- token weights -----------------------------------------------------------------
@pytest.mark.parametrize("hq,ps", [(16, 16), (16, 1), (32, 8), (32, 12)])
def test_a_token_of_great_weight_and_no_values(bsp, hq, ps):
    """A first token that takes all but 2^-10 .. 2^-36 of the softmax and whose values are zero or nearly so: the outputs
    are those of the others."""
    b = workloads.paged_batch(301, [1, 1], [1500, 700], hq, 2, 128, ps, "bf16", extra_pages=2)
    k8, ke, v8, ve = cache8(b, 301, ke=(0, 0), ve=(-6, -6))
    rng = np.random.default_rng(301)
    k8[:] = torch.from_numpy(rng.standard_normal(k8.shape)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    # a query of c in every dimension: the first token's score is 8 * 128 c / sqrt(128) / ln 2 = 130.6 c, the others'
    # N(0, 1.44 c)
    gaps = np.array([10, 14, 18, 22, 24, 26, 30, 36])[np.arange(hq) % 8]
    b.q = torch.from_numpy(np.broadcast_to((gaps / 130.6)[None, :, None], b.q.shape).copy()).bfloat16()
    for r in range(2):
        first = b.kv_indices[b.kv_indptr[r]]
        k8[first, 0] = 0x50  # 8
        v8[first, 0] = 0
        v8[first, 0, :, 64:] = 0x01  # 2^-9, the least code
    check_decode(bsp, b, [k8, ke, v8, ve], num_ctas=7)


# ---- queries -----------------------------------------------------------------------
@pytest.mark.parametrize("by", [-100, -40, -20, 20, 40, 80])
@pytest.mark.parametrize("hq,ps,cap", [(16, 16, 0.0), (32, 16, 0.0), (16, 1, 30.0), (32, 5, 0.0)])
def test_queries_of_any_size(bsp, hq, ps, cap, by):
    """q * 2^by over keys with exponents lower by as much: the same scores, the same bits."""
    b = workloads.paged_batch(302, [1, 1, 1], [900, 77, 3], hq, 2, 128, ps, "bf16", extra_pages=1)
    b.soft_cap = cap
    k8, ke, v8, ve = cache8(b, 302)
    used = np.unique(b.kv_indices)
    want = check_decode(bsp, b, [k8, ke, v8, ve], num_ctas=5)
    b.q = b.q * 2.0 ** by
    ke = ke.copy()
    ke[used] -= by
    got = check_decode(bsp, b, [k8, ke, v8, ve], num_ctas=5)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("hq", [16, 32])
def test_heads_of_different_sizes(bsp, hq):
    """Rows of q from 2^-60 to 2^60, with a dimension far above the row's others, over keys near 1, and rows of zeros."""
    b = workloads.paged_batch(303, [1, 1], [600, 40], hq, 2, 128, 16, "bf16")
    c8 = cache8(b, 303)
    scale = 2.0 ** np.linspace(-60, 60, hq).round()
    q = b.q.float() * torch.from_numpy(scale).float()[None, :, None]
    q[:, ::3, 5] *= 2.0 ** 14
    q[1, hq // 2] = 0
    b.q = q.bfloat16()
    check_decode(bsp, b, c8, num_ctas=5)


def test_subnormal_queries(bsp):
    """bf16 values below the normal range, the largest of their row."""
    b = workloads.paged_batch(304, [1], [300], 8, 1, 128, 16, "bf16")
    k8, ke, v8, ve = cache8(b, 304)
    b.q = (b.q.float() * 2.0 ** -129).bfloat16()
    used = np.unique(b.kv_indices)
    ke[used] = 118
    check_decode(bsp, b, [k8, ke, v8, ve], num_ctas=2)


# ---- what no head sees -------------------------------------------------------------
@pytest.mark.parametrize("hq,ps", [(16, 16), (32, 64), (16, 100), (32, 1)])
def test_nan_codes_before_the_window(bsp, hq, ps):
    """The page that the window begins in holds older tokens: their NaN codes reach nobody."""
    b = workloads.paged_batch(306, [1, 1, 1], [900, 77, 250], hq, 2, 128, ps, "bf16", extra_pages=1)
    b.window_left = 55
    c8 = cache8(b, 306)
    want = check_decode(bsp, b, c8, num_ctas=4)
    for r, n in enumerate((900, 77, 250)):
        for t in range(n - 1 - 55):
            page = b.kv_indices[b.kv_indptr[r] + t // ps]
            c8[0][page, t % ps] = c8[2][page, t % ps] = 0x7f
    got = check_decode(bsp, b, c8, num_ctas=4)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# ---- NaN ---------------------------------------------------------------------------
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("mode", ["decode", "prefill"])
def test_a_query_that_is_not_finite(bsp, mode, bad):
    """It reaches its own row alone, split (the first request) or not."""
    qo = [1, 1] if mode == "decode" else [9, 5]
    b = workloads.paged_batch(305, qo, [3000, 40], 16, 2, 128, 16, "bf16", causal=mode == "prefill")
    c8 = cache8(b, 305)
    want = run_block(bsp, b, c8, num_ctas=7)
    b.q = b.q.clone()
    last = len(b.q) - 1
    b.q[0, 3, 7] = b.q[last, 12, 100] = bad
    got = run_block(bsp, b, c8, num_ctas=7)
    for r, h in ((0, 3), (last, 12)):
        assert torch.isnan(got[0][r, h]).all() and torch.isnan(got[1][r, h])
        for t in want[:2] + got[:2]:
            t[r, h] = 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("mode", ["decode", "prefill"])
@pytest.mark.parametrize("ps", [16, 12])
def test_a_nan_key(bsp, mode, ps):
    """Its codes reach the rows of its request and kv head that see it: outputs and LSE, in a split request, one that is
    not split, and one that has no other key."""
    qo, kv = ([1] * 4, [3000, 40, 1, 77]) if mode == "decode" else ([9, 5, 1, 20], [3000, 40, 1, 77])
    b = workloads.paged_batch(307, qo, kv, 16, 2, 128, ps, "bf16", causal=mode == "prefill")
    c8 = cache8(b, 307)
    want = run_block(bsp, b, c8, num_ctas=9)
    hit = torch.zeros(want[1].shape, dtype=torch.bool)
    for r, (t, h) in enumerate(((1501, 1), (37, 0), (0, 1))):
        c8[0][b.kv_indices[b.kv_indptr[r] + t // ps], t % ps, h, 5] = 0x7f
        first = max(0, t - (kv[r] - qo[r]))  # the request's first position that sees token t
        hit[b.qo_indptr[r] + first:b.qo_indptr[r + 1], 8 * h:8 * h + 8] = True
    got = run_block(bsp, b, c8, num_ctas=9)
    hit = hit.cuda()
    assert torch.isnan(got[0][hit]).all() and torch.isnan(got[1][hit]).all()
    assert torch.equal(got[0][~hit], want[0][~hit]) and torch.equal(got[1][~hit], want[1][~hit])


# ---- ordinary batches within the row-wise bounds -----------------------------------
@pytest.mark.parametrize("case", DECODE, ids=[f"d{c[0]}" for c in DECODE])
def test_decode_rows(bsp, case):
    seed, kv, hq, hk, ps, C, w, cap = case
    b = workloads.paged_batch(seed, [1] * len(kv), kv, hq, hk, 128, ps, "bf16", extra_pages=3)
    b.window_left, b.soft_cap = w, cap
    check_decode(bsp, b, cache8(b, seed), num_ctas=C)


@pytest.mark.parametrize("ps", [1, 16])
def test_exponents_far_apart_rows(bsp, ps):
    b = workloads.paged_batch(231, [1, 1], [900, 77], 16, 2, 128, ps, "bf16", extra_pages=1)
    check_decode(bsp, b, cache8(b, 231, ke=(-25, -5), ve=(-70, 50)), num_ctas=7)


def test_full_size_rows(bsp):
    """64 requests of up to 8192 tokens."""
    b = workloads.batched_decode_bf16()
    check_decode(bsp, b, cache8(b, 237))


@pytest.mark.parametrize("ve", [(-117, -117), (-117, -100), (105, 108)])
@pytest.mark.parametrize("ps", [1, 16])
def test_exponents_at_the_ends(bsp, ps, ve):
    """V values next to the ends of fp32's range (the sums of 1500 of them still within it): the outputs' factor,
    2^(e - 15) of the running maxima, leaves the normal range at the low end and keeps 17 bits."""
    b = workloads.paged_batch(308, [1, 1], [1500, 70], 16, 2, 128, ps, "bf16", extra_pages=1)
    check_decode(bsp, b, cache8(b, 308, ve=ve), num_ctas=7)
