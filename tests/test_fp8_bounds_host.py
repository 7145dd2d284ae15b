"""The row-wise bounds of fp8_bounds.py are tight enough to notice a mistake: outputs of a wrong decode, computed here,
fail the check that the right ones pass."""
import numpy as np
import pytest
import torch

import oracle
import workloads
from fp8_bounds import check, decode_bounds
from oracle import fp8
from oracle import kv_cache as kc
from test_gpu_fp8_block import cache8


def make(kv, hq, hk, ps):
    b = workloads.paged_batch(311, [1] * len(kv), kv, hq, hk, 128, ps, "bf16", extra_pages=3)
    c8 = cache8(b, 311)
    k, v = kc.values(c8[0], c8[1]), kc.values(c8[2], c8[3])
    O, L = oracle.attention_of(b, k=k, v=v)
    A, _ = oracle.attention_of(b, k=k, v=np.abs(v))
    return b, c8, O, L, decode_bounds(b, k, fp8.dequantize(c8[2], 1.0), c8[3], O, L, A)


@pytest.fixture(scope="module", params=[([8192, 300], 32, 8, 16), ([5000, 33, 129], 32, 8, 8), ([1500, 3], 32, 2, 4),
                                        ([700, 1, 3000], 32, 8, 1)], ids=["page16", "page8", "page4", "page1"])
def case(request):
    oracle.build()
    return make(*request.param)


def to_bf16(x):
    return torch.from_numpy(x).bfloat16().double().numpy()


def rejected(o, l, O, L, bounds):
    with pytest.raises(AssertionError):
        check(o, l, O, L, *bounds)


def test_right_outputs_pass(case):
    b, c8, O, L, bounds = case
    check(to_bf16(O), L.astype(np.float32), O, L, *bounds)


def test_few_elements_would_pass_as_zero(case):
    b, c8, O, L, bounds = case
    assert (np.abs(O) <= bounds[0]).mean() < 0.05
    rejected(np.zeros_like(O), L, O, L, bounds)


# What can be seen: n tokens of equal weight 1 / n among which m get values wrong by half move an element by about
# sqrt(m) / n, against a bound of 2^-11 of the mean |value|: m = 16 up to n of about 8000. K moves LSE by m / n of the
# scores' variance, against about 2^-12.
@pytest.mark.parametrize("by", [-1, 1])
@pytest.mark.parametrize("which", [1, 3], ids=["K", "V"])
def test_pages_with_a_wrong_exponent(case, which, by):
    """128 neighbouring tokens in the middle of the longest request, one kv head, off by one."""
    b, c8, O, L, bounds = case
    r = int(np.argmax(b.kv_lens))
    i = int(b.kv_indptr[r] + b.kv_indptr[r + 1]) // 2
    bad = [a.copy() for a in c8]
    bad[which][b.kv_indices[i:i + 128 // b.page_size], 1] += by
    o, l = oracle.attention_of(b, k=kc.values(bad[0], bad[1]), v=kc.values(bad[2], bad[3]))
    rejected(to_bf16(o), l, O, L, bounds)


@pytest.mark.parametrize("by", [-1, 1])
@pytest.mark.parametrize("which", [1, 3], ids=["K", "V"])
def test_one_page_with_a_wrong_exponent(which, by):
    """Of 63 pages."""
    oracle.build()
    b, c8, O, L, bounds = make([1000, 300], 32, 8, 16)
    bad = [a.copy() for a in c8]
    bad[which][b.kv_indices[31], 1] += by
    o, l = oracle.attention_of(b, k=kc.values(bad[0], bad[1]), v=kc.values(bad[2], bad[3]))
    rejected(to_bf16(o), l, O, L, bounds)


def test_lost_tokens(case):
    """Sixteen tokens (or one page) of the longest request not read."""
    b, c8, O, L, bounds = case
    r = int(np.argmax(b.kv_lens))
    i = int(b.kv_indptr[r] + b.kv_indptr[r + 1]) // 2
    bad = [a.copy() for a in c8]
    for page in b.kv_indices[i:i + max(1, 16 // b.page_size)]:
        bad[2][page] = 0
    o, _ = oracle.attention_of(b, k=kc.values(bad[0], bad[1]), v=kc.values(bad[2], bad[3]))
    rejected(to_bf16(o), L, O, L, bounds)
