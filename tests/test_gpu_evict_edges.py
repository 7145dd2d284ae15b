"""Gathered weights beside requests that hold NaN."""
import numpy as np
import pytest
import torch

import workloads
from gpu_helpers import lib
from oracle import evict as ev
from oracle import kv_cache as kc
from test_gpu_evict import F8, dev, table, true_lse, values
from test_gpu_fp8_block import cache8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bsp():
    return lib()


@pytest.mark.parametrize("ps", [1, 5, 16, 128])
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "f32", "diff"])
@pytest.mark.parametrize("qo,kv", [([1] * 5, [700, 901, 40, 17, 333]), ([30, 5, 40, 17, 100], [700, 901, 40, 17, 333]),
                                   ([600, 300, 40, 640, 333], [700, 901, 40, 650, 333])], ids=["decode", "chunks", "prompts"])
def test_a_request_of_nan_reaches_no_other(bsp, ps, kind, qo, kv):
    """Keys, queries and LSE of one request are NaN: its weights are, and every bit of the others' stays."""
    if kind == "f32" and max(qo) > 100:
        qo, kv = [20, 5, 40, 17, 60], [100, 901, 40, 17, 60]
    b = workloads.paged_batch(96, qo, kv, 16, 4, 128, ps, "f32" if kind == "f32" else "bf16", causal=True, extra_pages=2)
    ke, lam = None, torch.full((16,), 0.7, device="cuda") if kind == "diff" else None
    scale = 128 ** -0.5
    if kind == "e4m3":
        codes, e, _, _ = cache8(b, 96)
        k, kt, ke = kc.values(codes, e), dev(codes).view(F8), dev(e)
    else:
        k, kt = values(b.k_pages), b.k_pages.cuda()
    lse = dev(true_lse(b, k, scale, -1, 0.0, 2 if lam is not None else 1))
    w0 = torch.rand(kt.shape[0], 4, ps, device="cuda")
    t, qi = table(b), dev(b.qo_indptr.astype(np.int32))

    def run(q, lse, kt):
        w = w0.clone()
        bsp.accumulate_weights(q, lse, kt, w, *t, qo_indptr=qi, sm_scale=scale, decay=0.5, k_exp=ke, lam=lam)
        return w
    want = run(b.q.cuda(), lse, kt)
    for i in range(5):
        pg, pl = (torch.from_numpy(x).cuda() for x in ev.slots(b.kv_indptr, b.kv_indices, i, kv[i], ps))
        its = slice(int(b.qo_indptr[i]), int(b.qo_indptr[i + 1]))
        q, l, x = b.q.cuda(), lse.clone(), kt.clone()
        q[its], l[its] = float("nan"), float("nan")
        if kind == "e4m3":
            x.view(torch.uint8)[pg, pl] = 0x7f
        else:
            x[pg, pl] = float("nan")
        got = run(q, l, x)
        torch.cuda.synchronize()
        assert torch.isnan(got[pg, :, pl]).all()
        got[pg, :, pl] = want[pg, :, pl]
        assert torch.equal(got, want), i
