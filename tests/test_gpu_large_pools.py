"""Differential attention, gathered weights, the choice and the move at the far end of pools of more than 2^32 bytes: the same
bits as in a pool that holds these pages alone."""
import numpy as np
import pytest
import torch

import workloads
from gpu_helpers import lib
from test_gpu_evict import F8, dev
from test_gpu_fp8_block import cache8

pytestmark = pytest.mark.gpu
H, PS = 8, 16


@pytest.fixture(scope="module")
def bsp():
    return lib()


def far(t, pages):
    """t [n, ...] as the last of `pages` pages."""
    big = torch.empty((pages,) + tuple(t.shape[1:]), dtype=t.dtype, device="cuda")
    big[pages - t.shape[0]:].view(torch.uint8).copy_(t.view(torch.uint8))
    return big


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("qo", [[1, 1, 1], [200, 64, 33]], ids=["decode", "prefill"])
def test_far_pages(bsp, kind, qo):
    row = {"bf16": 256, "e4m3": 128, "f32": 512}[kind]
    pages = int(1.1 * 2 ** 32) // (row * H * PS)
    b = workloads.paged_batch(95, qo, [700, 64, 300], 16, H, 128, PS, "f32" if kind == "f32" else "bf16", causal=True)
    if kind == "e4m3":
        k, ke, v, ve = (dev(x) for x in cache8(b, 95))
        pools, exps = [k.view(F8), v.view(F8)], [ke, ve]
    else:
        pools, exps = [b.k_pages.cuda(), b.v_pages.cuda()], [None, None]
    n = pools[0].shape[0]
    q, lam = b.q.cuda(), torch.full((16,), 0.7, device="cuda")
    indptr, last, qi = (dev(x.astype(np.int32)) for x in (b.kv_indptr, b.last_page_len, b.qo_indptr))
    w0, budget = torch.rand(n, H, PS, device="cuda"), dev(np.array([300, 20, 150], np.int32))
    decode = max(qo) == 1

    def serve(k, v, ke, ve, w, indices):
        """The differential run (fp32 pools: a given LSE), its weights, the choice and the move."""
        out = []
        if kind == "f32":
            lse = torch.full(q.shape[:2], 6.0, device="cuda")
            bsp.accumulate_weights(q, lse, k, w, indptr, indices, last, qo_indptr=qi)
        else:
            pa = bsp.PagedAttention("decode" if decode else "prefill", 16, H, 128, PS, True, max_batch=3, max_qo_tokens=int(sum(qo)),
                                    differential=True)
            pa.plan(b.kv_indptr, b.last_page_len, qo_indptr=None if decode else b.qo_indptr)
            o, lse = pa.run_differential(q, k, v, indices, lam, k_exp=ke, v_exp=ve)
            assert pa.check_device_error() == 0
            out = [o, lse]
            bsp.accumulate_weights(q, lse, k, w, indptr, indices, last, qo_indptr=qi, lam=lam, k_exp=ke)
        kept, new = bsp.select_tokens(w, indptr, indices, last, budget, 300)
        bsp.compact_cache(kept, new, indptr, indices, last, k, v, weights=w, k_exp=ke, v_exp=ve)
        return [x.clone() for x in out + [kept, new] + [t[-n:] for t in (k, v, w, ke, ve) if t is not None]]
    ids = dev(b.kv_indices.astype(np.int32))
    big = [far(t, pages) if t is not None else None for t in (pools[0], pools[1], *exps, w0)]
    want = serve(*(t.clone() if t is not None else None for t in (*pools, *exps)), w0.clone(), ids)
    got = serve(*big, ids + (pages - n))
    torch.cuda.synchronize()
    assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(got, want))
