"""Gathered weights where a wait inside the kernels gives up: nothing keeps an old weight unnoticed. (The self-test's call: the
warps that bring the keys stop after the first few, the others' waits end after about a millisecond.)"""
import ctypes

import numpy as np
import pytest
import torch

import workloads
from gpu_helpers import lib
from test_gpu_evict import F8, dev, table, true_lse, values
from test_gpu_fp8_block import cache8
from oracle import evict as ev
from oracle import kv_cache as kc

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bsp():
    return lib()


CASES = {  # queries and keys per request
    "decode": ([1] * 8, [3000] * 8), "e4m3": ([1] * 8, [3000] * 8),       # about 20 tasks per CTA
    "prompts": ([64, 40] * 30, [700, 900] * 30),                          # several units per CTA, one or two tiles each
    "long": ([1100, 1500], [1300, 1500])}                                 # a unit per CTA, many tiles


@pytest.mark.parametrize("kind", CASES)
def test_a_wait_that_gives_up_leaves_nan(bsp, kind):
    from block_sparse_paged_gb300 import _native as N
    qo, kv = CASES[kind]
    b = workloads.paged_batch(81, qo, kv, 16, 4, 128, 16, "bf16", causal=True, extra_pages=3)
    scale, ke = 128 ** -0.5, None
    if kind == "e4m3":
        codes, e, _, _ = cache8(b, 81)
        k, kt, ke = kc.values(codes, e), dev(codes).view(F8), dev(e)
    else:
        k, kt = values(b.k_pages), b.k_pages.cuda()
    lse = dev(true_lse(b, k, scale, -1, 0.0, 1))
    q, qi, t = b.q.cuda(), dev(b.qo_indptr.astype(np.int32)), table(b)
    w0 = torch.rand(kt.shape[0], 4, 16, device="cuda") + 1.0

    def good():
        w = w0.clone()
        bsp.accumulate_weights(q, lse, kt, w, *t, qo_indptr=qi, sm_scale=scale, decay=0.5, k_exp=ke)
        return w
    want, w = good(), w0.clone()
    p = lambda x: None if x is None else ctypes.c_void_p(x.data_ptr())  # noqa: E731
    problem = N.Problem(N.BSP_MODE_DECODE, 16, 4, 128, 16, 1, N.BSP_DTYPE_BF16, -1, 0.0)
    N.check(N.load().bsp_check_weights_wait(ctypes.byref(problem), p(q), p(lse), q.shape[0], p(kt), p(ke), kt.shape[0], p(w), b.batch,
                                            p(qi), p(t[0]), p(t[1]), t[1].numel(), p(t[2]), scale, 0.5, 2_000_000,
                                            ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)))
    torch.cuda.synchronize()
    used = np.zeros(w.shape, bool)
    for i, L in enumerate(kv):
        pg, pl = ev.slots(b.kv_indptr, b.kv_indices, i, L, 16)
        used[pg, :, pl] = True
    got, right, old = (x.cpu().numpy() for x in (w, want, w0))
    nan = np.isnan(got)
    assert not np.isnan(right).any() and nan[used].any() and not nan[used].all()
    assert (nan | (got == right))[used].all() and np.array_equal(got[~used], old[~used])
    assert torch.equal(good(), want)
