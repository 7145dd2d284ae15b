"""Windowed prefill over the 8-bit cache: what stands before the windows."""
import ctypes

import numpy as np
import pytest
import torch

import workloads
from block_sparse_paged_gb300 import _native as N
from gpu_helpers import lib
from test_gpu_fp8_block import cache8, check, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bsp():
    return lib()


@pytest.mark.parametrize("region", [False, True], ids=["inside", "copied"])
@pytest.mark.parametrize("ps,qo", [(5, [31, 5, 40]), (12, [31, 5, 40]), (16, [31, 5, 40]), (128, [200, 5, 40])])
def test_nan_codes_before_the_window_of_prompts(bsp, ps, qo, region):
    """The page that a window begins in holds older tokens: NaN codes that no row of a tile sees reach none, converted inside
    the kernel or copied first."""
    kv, window = [700, 900, 40], 51
    b = workloads.paged_batch(308, qo, kv, 16, 4, 128, ps, "bf16", causal=True, extra_pages=1)
    b.window_left = window
    c8 = cache8(b, 308)
    pa = bsp.PagedAttention("prefill", 16, 4, 128, ps, True, max_batch=3, max_qo_tokens=sum(qo), window_left=window, num_ctas=2)
    pa.plan(b.kv_indptr, b.last_page_len, qo_indptr=b.qo_indptr)
    q, idx = b.q.cuda(), torch.from_numpy(b.kv_indices.astype(np.int32)).cuda()
    n = len(b.kv_indices) * ps * 4 * 512 if region else 0
    buf = torch.empty(n, dtype=torch.uint8, device="cuda") if region else None
    p = lambda t: None if t is None else ctypes.c_void_p(t.data_ptr())  # noqa: E731

    def run():
        k, ke, v, ve = (torch.from_numpy(a).cuda() for a in c8)
        out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
        N.check(N.load().bsp_prefill_run_fp8_block(
            ctypes.byref(pa.info), p(q), p(k), p(v), p(ke), p(ve), p(idx), k.shape[0], 128 ** -0.5, p(out), p(lse), p(buf), n,
            p(pa.workspace), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)))
        torch.cuda.synchronize()
        assert pa.check_device_error() == 0
        return out, lse
    want = run()
    check(*want, reference(b, c8), 2.0 ** -8, b)
    for r in range(3):
        for t in range(kv[r] - qo[r] - window):
            page = b.kv_indices[b.kv_indptr[r] + t // ps]
            c8[0][page, t % ps] = c8[2][page, t % ps] = 0x7f
    got = run()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
