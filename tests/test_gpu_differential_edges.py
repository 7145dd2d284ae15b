"""Differential attention at the edges: norms of rows that are zero, queries of NaN, values before a window and of other requests, the
order of a queue's items."""
import numpy as np
import pytest
import torch

from gpu_helpers import lib
from oracle import evict as ev
from test_gpu_differential import Run

pytestmark = pytest.mark.gpu
MODES = pytest.mark.parametrize("mode", ["decode", "prefill"])
POOLS = pytest.mark.parametrize("f8", [False, True], ids=["bf16", "e4m3"])


@pytest.fixture(scope="module")
def bsp():
    return lib()


def sizes(mode):
    """Requests without keys, with one, and with fewer keys than queries; outputs on one CTA and split."""
    return ([1, 1, 1], [0, 1, 700]) if mode == "decode" else ([3, 70, 200], [0, 5, 700])


@MODES
@POOLS
@pytest.mark.parametrize("num_ctas", [1, 40])
def test_norm_of_rows_without_keys(bsp, mode, f8, num_ctas):
    """A query without a visible key gets 0, its norm's eps being 0 too."""
    qo, kv = sizes(mode)
    r = Run(bsp, 71, qo, kv, 16, 4, 16, mode=mode, f8=f8, norm=True, num_ctas=num_ctas)
    out, lse = r(norm_eps=0.0)
    torch.cuda.synchronize()
    got, none = out.float().cpu().numpy(), np.isneginf(lse.cpu().numpy()).all(axis=2)
    rows = sum(max(0, q - k) for q, k in zip(qo, kv))
    assert none.sum() == 16 * rows and (got[none] == 0).all() and np.isfinite(got).all()
    r.check(*r())


@MODES
@POOLS
def test_norm_of_maps_that_cancel(bsp, mode, f8):
    """Equal maps and lambda 1: 0 over sqrt(0 + 0) is 0."""
    r = Run(bsp, 72, [1, 1] if mode == "decode" else [50, 9], [300, 40], 16, 4, 16, mode=mode, f8=f8, lam=1.0, norm=True)
    r.q[..., 64:] = r.q[..., :64]
    r.k.view(torch.uint8 if f8 else torch.bfloat16)[..., 64:] = r.k.view(torch.uint8 if f8 else torch.bfloat16)[..., :64]
    assert (r(norm_eps=0.0, return_lse=False) == 0).all()


@MODES
@POOLS
@pytest.mark.parametrize("num_ctas", [1, 40])
def test_nan_queries_make_nan(bsp, mode, f8, num_ctas):
    """A query of NaN has outputs and LSE of NaN, its output on one CTA or split over several; the other heads stay."""
    qo, kv = ([1, 1], [900, 700]) if mode == "decode" else ([70, 5], [900, 700])
    r = Run(bsp, 75, qo, kv, 16, 4, 16, mode=mode, f8=f8, num_ctas=num_ctas)
    want, wl = (x.clone() for x in r())
    r.q[1, 3] = float("nan")
    out, lse = r()
    torch.cuda.synchronize()
    assert torch.isnan(out[1, 3]).all() and torch.isnan(lse[1, 3]).all()
    out[1, 3], lse[1, 3] = want[1, 3], wl[1, 3]
    assert torch.equal(out, want) and torch.equal(lse, wl)


@MODES
@pytest.mark.parametrize("num_ctas", [1, 40])
def test_one_map_of_nan(bsp, mode, num_ctas):
    """NaN in the second half of a query alone: the first map's LSE stays."""
    qo, kv = ([1, 1], [900, 700]) if mode == "decode" else ([70, 5], [900, 700])
    r = Run(bsp, 76, qo, kv, 16, 4, 16, mode=mode, num_ctas=num_ctas)
    want, wl = (x.clone() for x in r())
    r.q[1, 3, 64:] = float("nan")
    out, lse = r()
    torch.cuda.synchronize()
    assert torch.isnan(out[1, 3]).all() and torch.isnan(lse[1, 3, 1]) and torch.equal(lse[1, 3, 0], wl[1, 3, 0])
    out[1, 3], lse[1, 3] = want[1, 3], wl[1, 3]
    assert torch.equal(out, want) and torch.equal(lse, wl)


@pytest.mark.parametrize("norm", [False, True], ids=["plain", "norm"])
def test_items_without_keys_behind_split_ones(bsp, norm):
    """Queues with a final output, then a partial state of one tile, then an output without keys, which writes none of what the
    warps trade for the first: the same bits every time."""
    r = Run(bsp, 77, [32] * 8 + [2] * 2 + [20] * 8, [60] * 8 + [500] * 2 + [0] * 8, 4, 1, 16, mode="prefill", num_ctas=8, chunks_per_cta=2,
            norm=norm)
    queue, items, _ = r.pa.plan_arrays()

    def kind(w):
        keys = w["kv_end"] - w["kv_start"]
        return "none" if keys == 0 else "final" if w["slot"] < 0 else "tile" if keys <= 128 else "tiles"
    of = [[kind(w) for w in items[a:b]] for a, b in zip(queue, queue[1:])]
    assert any(q[i:i + 3] == ["final", "tile", "none"] for q in of for i in range(len(q)))
    out, lse = (x.clone() for x in r())
    r.check(out, lse)
    for _ in range(50):
        o, l = r()
        assert torch.equal(o, out) and torch.equal(l, lse)


@MODES
@POOLS
def test_replay_after_another_plan(bsp, mode, f8):
    """A captured run follows a new plan in its workspace, and sets no status there."""
    qo, kv = ([1] * 3, [700, 20, 300]) if mode == "decode" else ([200, 20, 1], [700, 20, 300])
    r = Run(bsp, 78, qo, kv, 16, 4, 16, mode=mode, f8=f8, norm=True, max_gather_pages=100 if mode == "prefill" else 0)
    r()
    out, lse = torch.empty_like(r.q), torch.empty(r.q.shape[:2] + (2,), device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r(out=out, lse=lse)
    n = Run(bsp, 79, [1] * 3 if mode == "decode" else [100, 100, 21], [300, 600, 90], 16, 4, 16, mode=mode, f8=f8, norm=True)
    pool, tab = n.k.shape[0], n.idx.numel()
    assert n.q.shape == r.q.shape and pool <= r.k.shape[0] and tab <= r.idx.numel()
    r.pa.plan(n.b.kv_indptr, n.b.last_page_len, qo_indptr=n.b.qo_indptr)
    for mine, its in [(r.k.view(torch.uint8), n.k.view(torch.uint8)), (r.v.view(torch.uint8), n.v.view(torch.uint8)),
                      (r.idx, n.idx)] + [(r.e[x], n.e[x]) for x in r.e]:
        mine[:its.shape[0]] = its
    for mine, its in ((r.q, n.q), (r.lam_t, n.lam_t), (r.norm_t, n.norm_t)):
        mine.copy_(its)
    graph.replay()
    n.pa = r.pa  # (whose status word `check` asks)
    n.check(out, lse)


@MODES
@POOLS
@pytest.mark.parametrize("num_ctas", [1, 40])
@pytest.mark.parametrize("ps,window", [(1, 50), (5, 51), (12, 300), (16, 50), (128, 303)])
def test_values_before_a_window_reach_nobody(bsp, mode, f8, num_ctas, ps, window):
    """The page that a window begins in holds older tokens: NaN of theirs changes no bit."""
    qo, kv = ([1, 1, 1], [700, 900, 40]) if mode == "decode" else ([31, 5, 40], [700, 900, 40])
    r = Run(bsp, 80, qo, kv, 16, 4, ps, mode=mode, f8=f8, window=window, num_ctas=num_ctas)
    out, lse = (x.clone() for x in r())
    r.check(out, lse)
    for i, (n, L) in enumerate(zip(qo, kv)):
        if L - n - window > 0:
            pg, pl = (torch.from_numpy(x).cuda() for x in ev.slots(r.b.kv_indptr, r.b.kv_indices, i, L - n - window, ps))
            for t in (r.k, r.v):
                if f8:
                    t.view(torch.uint8)[pg, pl] = 0x7f
                else:
                    t[pg, pl] = float("nan")
    o, l = r()
    torch.cuda.synchronize()
    assert torch.equal(o, out) and torch.equal(l, lse)


@MODES
@POOLS
@pytest.mark.parametrize("num_ctas", [1, 40])
@pytest.mark.parametrize("ps", [1, 5, 8, 16, 128])
def test_a_request_of_nan_reaches_no_other(bsp, mode, f8, num_ctas, ps):
    """K and V of one request are NaN: its outputs are, and every bit of the others' stays."""
    qo, kv = ([1] * 5, [700, 901, 40, 17, 333]) if mode == "decode" else ([30, 5, 40, 17, 100], [700, 901, 40, 17, 333])
    r = Run(bsp, 82, qo, kv, 16, 4, ps, mode=mode, f8=f8, num_ctas=num_ctas)
    out, lse = (x.clone() for x in r())
    r.check(out, lse)
    clean = [t.clone() for t in (r.k, r.v)]
    for i in range(5):
        for t, c in zip((r.k, r.v), clean):
            t.view(torch.uint8).copy_(c.view(torch.uint8))
        pg, pl = (torch.from_numpy(x).cuda() for x in ev.slots(r.b.kv_indptr, r.b.kv_indices, i, kv[i], ps))
        for t in (r.k, r.v):
            if f8:
                t.view(torch.uint8)[pg, pl] = 0x7f
            else:
                t[pg, pl] = float("nan")
        o, l = r()
        torch.cuda.synchronize()
        its = slice(int(r.b.qo_indptr[i]), int(r.b.qo_indptr[i + 1]))
        assert torch.isnan(o[its]).all() and torch.isnan(l[its]).all()
        o[its], l[its] = out[its], lse[its]
        assert torch.equal(o, out) and torch.equal(l, lse), i
