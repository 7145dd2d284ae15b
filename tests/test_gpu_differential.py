"""Differential attention on the GPU against the plain 64-bit form (oracle.evict.differential). The bounds are derived beside
`check`."""
import numpy as np
import pytest
import torch

import workloads
from gpu_helpers import lib
from oracle import evict as ev
from oracle import kv_cache as kc
from test_gpu_fp8_block import cache8

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def bsp():
    return lib()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Run:
    """One problem: its plan's object, device tensors and a call."""

    def __init__(self, bsp, seed, qo, kv, Hq, H, ps, mode=None, f8=False, window=-1, cap=0.0, norm=False, out_scale=1.0, num_ctas=None,
                 lam=None, **kw):
        decode = mode == "decode" if mode else max(qo, default=0) <= 1
        self.b = b = workloads.paged_batch(seed, qo, kv, Hq, H, 128, ps, "bf16", causal=not decode, extra_pages=3)
        rng = np.random.default_rng(seed)
        self.decode, self.f8, self.window, self.cap, self.out_scale = decode, f8, window, cap, out_scale
        self.pa = bsp.PagedAttention("decode" if decode else "prefill", Hq, H, 128, ps, causal=True, max_batch=max(1, len(qo)),
                                     max_qo_tokens=max(1, int(np.sum(qo))), window_left=window, logits_soft_cap=cap, num_ctas=num_ctas,
                                     differential=True, **kw)
        self.pa.plan(b.kv_indptr, b.last_page_len, qo_indptr=b.qo_indptr)
        self.lam = (0.8 + 0.3 * rng.standard_normal(Hq)).astype(np.float32) if lam is None else np.full(Hq, lam, np.float32)
        self.norm = (1 + 0.2 * rng.standard_normal(128)).astype(np.float32) if norm else None
        self.e = {}
        if f8:
            c = cache8(b, seed)
            self.k64, self.v64 = kc.values(c[0], c[1]), kc.values(c[2], c[3])
            self.k, self.v = dev(c[0]).view(F8), dev(c[2]).view(F8)
            self.e = dict(k_exp=dev(c[1]), v_exp=dev(c[3]))
        else:
            self.k64, self.v64 = b.k_pages.double().numpy(), b.v_pages.double().numpy()
            self.k, self.v = b.k_pages.cuda(), b.v_pages.cuda()
        self.q, self.idx, self.lam_t = b.q.cuda(), dev(b.kv_indices.astype(np.int32)), dev(self.lam)
        self.norm_t = None if self.norm is None else dev(self.norm)

    def __call__(self, **kw):
        return self.pa.run_differential(self.q, self.k, self.v, self.idx, self.lam_t, norm_weight=self.norm_t, out_scale=self.out_scale,
                                        **self.e, **kw)

    def check(self, out, lse):
        """Bounds. A score is 1/8 of a sum of 64 products in fp32 (2^-23 per addition, tensor cores may cut) and scaled, moved by
        its maximum and exponentiated: off by e = s 64 2^-23 + 4 s 2^-23 + 2^-20 at most, s >= sum |q k| / 8; capped ones by 2^-21
        cap more. So LSE is off by e + 2^-22 |LSE|, and a map's output by (P |v|) (e + r), r = 2^-8 for P in bf16, 2^-11 in f16
        (8-bit decode), both + 2^-20 for the sums; y adds up over the maps; the norm's factor is off by |dy| / |y| relatively; the
        output is rounded once: 2^-8."""
        torch.cuda.synchronize()
        assert self.pa.check_device_error() == 0
        b, q = self.b, self.b.q.double().numpy()
        o, z, size = ev.differential(q, np.nan_to_num(self.k64), np.nan_to_num(self.v64), b.qo_indptr, b.kv_indptr, b.kv_indices,
                                     b.last_page_len, 0.125, self.lam.astype(np.float64),
                                     None if self.norm is None else self.norm.astype(np.float64), 1e-5, self.out_scale, self.window, self.cap)
        s = 0.125 * np.abs(q).sum(axis=2).max(initial=0.0) * np.nanmax(np.abs(self.k64), initial=0.0)
        e = s * 68 * 2.0 ** -23 + 2.0 ** -20 + self.cap * 2.0 ** -21
        got, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
        fin = np.isfinite(z)
        assert np.array_equal(np.isneginf(l), ~fin)
        assert (np.abs(l[fin] - z[fin]) <= e + 2.0 ** -22 * np.abs(z[fin])).all(), np.abs(l[fin] - z[fin]).max()
        d = size * (e + (2.0 ** -11 if self.f8 and self.decode else 2.0 ** -8) + 2.0 ** -20)
        tol = d + 2.0 ** -8 * (np.abs(o) + d) + 2.0 ** -130
        if self.norm is not None:  # |y| of a row, from the output without its weights
            w = np.where(self.norm == 0, 1.0, np.abs(self.norm))
            rel = np.linalg.norm(d / w, axis=2) / np.maximum(np.linalg.norm(o / w, axis=2), 1e-300)
            tol = tol + np.abs(o) * (rel / np.maximum(1 - rel, 0.1))[:, :, None]
        assert np.isfinite(got).all()
        worst = (np.abs(got - o) - tol).max(initial=-1.0)
        assert worst <= 0, (worst, np.abs(got - o).max())
        return got


DECODE = [  # kv lengths, Hq, H, ps
    ([1, 0, 70, 300, 1500], 32, 8, 16), ([64, 63, 65, 128, 129], 8, 8, 1), ([333], 8, 1, 64), ([5, 900], 15, 5, 5),
    ([2000, 1], 24, 8, 12), ([129, 127], 4, 2, 128), ([77, 300], 14, 2, 8)]


@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("norm", [False, True], ids=["plain", "norm"])
@pytest.mark.parametrize("case", DECODE, ids=str)
def test_decode(bsp, case, norm, f8):
    kv, Hq, H, ps = case
    r = Run(bsp, 41, [1] * len(kv), kv, Hq, H, ps, f8=f8, norm=norm, out_scale=0.2 if norm else 1.0)
    r.check(*r())


@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("num_ctas", [3, 40, 304])
def test_decode_split_outputs(bsp, num_ctas, f8):
    """Chunks of one output on several CTAs, folded by the last of them; many queues per CTA. Again on the same plan: the same bits."""
    r = Run(bsp, 42, [1] * 6, [4000, 17, 900, 64, 7000, 2500], 32, 8, 16, f8=f8, norm=True, num_ctas=num_ctas, chunks_per_cta=2)
    a = r()
    r.check(*a)
    assert all(torch.equal(x, y) for x, y in zip(a, r()))


def test_decode_many_folds_of_one_cta(bsp):
    """One queue that completes more outputs than its list holds."""
    r = Run(bsp, 43, [1] * 30, [400] * 30, 8, 2, 16, num_ctas=1, chunks_per_cta=64, norm=True)
    assert r.pa.info.num_merges == 60  # chunks of 384 tokens
    r.check(*r())


@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("window,cap", [(1, 0.0), (60, 0.0), (700, 15.0), (-1, 5.0)])
def test_decode_variants(bsp, window, cap, f8):
    r = Run(bsp, 44, [1] * 4, [700, 33, 1, 1500], 16, 4, 16, f8=f8, window=window, cap=cap, norm=True)
    r.check(*r())


def test_decode_several_positions(bsp):
    r = Run(bsp, 45, [3, 0, 5], [40, 20, 900], 16, 4, 16, mode="decode", norm=True)
    r.check(*r())


PREFILL = [  # queries, kv lengths, Hq, H, ps
    ([100, 37, 1], [100, 300, 1], 32, 8, 16), ([70, 0, 5], [150, 40, 5], 8, 8, 1), ([129], [700], 64, 1, 64),
    ([257, 64], [257, 1000], 16, 2, 5), ([33, 128], [33, 128], 4, 4, 128), ([40, 300], [2000, 300], 32, 2, 12)]


@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("norm", [False, True], ids=["plain", "norm"])
@pytest.mark.parametrize("case", PREFILL, ids=str)
def test_prefill(bsp, case, norm, f8):
    qo, kv, Hq, H, ps = case
    r = Run(bsp, 46, qo, kv, Hq, H, ps, mode="prefill", f8=f8, norm=norm, out_scale=0.2 if norm else 1.0)
    r.check(*r())


@pytest.mark.parametrize("num_ctas", [1, 5, 152, 304])
@pytest.mark.parametrize("norm", [False, True], ids=["plain", "norm"])
def test_prefill_split_outputs(bsp, num_ctas, norm):
    """Items with final outputs and with partial states in one queue, in every order."""
    r = Run(bsp, 47, [60, 300, 5, 0, 64], [3000, 300, 2000, 10, 64], 16, 4, 16, num_ctas=num_ctas, norm=norm, chunks_per_cta=2)
    a = r()
    r.check(*a)
    assert all(torch.equal(x, y) for x, y in zip(a, r()))


@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("window,cap", [(1, 0.0), (100, 0.0), (300, 15.0), (-1, 5.0)])
def test_prefill_variants(bsp, window, cap, f8):
    r = Run(bsp, 48, [200, 77], [500, 77], 16, 4, 16, f8=f8, window=window, cap=cap, norm=True)
    r.check(*r())


def test_prefill_copy_regions(bsp):
    """Pages under 8 tokens copied first; the 8-bit cache into the workspace's region or a tensor of the call: the same bits."""
    a = Run(bsp, 49, [100, 30], [400, 90], 16, 4, 3, max_gather_pages=200)
    c = Run(bsp, 49, [100, 30], [400, 90], 16, 4, 3)
    a.check(*a())
    assert all(torch.equal(x, y) for x, y in zip(a(), c()))
    a = Run(bsp, 49, [100, 30], [400, 90], 16, 4, 16, f8=True, max_gather_pages=40)
    c = Run(bsp, 49, [100, 30], [400, 90], 16, 4, 16, f8=True)
    a.check(*a())
    assert all(torch.equal(x, y) for x, y in zip(a(), c()))


@pytest.mark.parametrize("mode", ["decode", "prefill"])
@pytest.mark.parametrize("lam", [0.0, 1.0, -2.5])
def test_lambda(bsp, mode, lam):
    """lam 0 is the first map's attention alone."""
    r = Run(bsp, 50, [1, 1] if mode == "decode" else [50, 9], [300, 40], 16, 4, 16, mode=mode, lam=lam)
    r.check(*r())


@pytest.mark.parametrize("mode", ["decode", "prefill"])
def test_equal_maps_cancel(bsp, mode):
    """Both halves equal and lam 1: the difference is exactly 0, and the norm of a zero row is 0, not NaN."""
    r = Run(bsp, 51, [1, 1] if mode == "decode" else [50, 9], [300, 40], 16, 4, 16, mode=mode, lam=1.0, norm=True)
    r.q[..., 64:] = r.q[..., :64]
    r.k[..., 64:] = r.k[..., :64]
    out, lse = r()
    assert (out == 0).all() and torch.equal(lse[..., 0], lse[..., 1])


@pytest.mark.parametrize("mode", ["decode", "prefill"])
@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "e4m3"])
def test_streams_graphs_and_given_outputs(bsp, mode, f8):
    qo, kv = ([1] * 3, [700, 20, 300]) if mode == "decode" else ([200, 20, 1], [700, 20, 300])
    r = Run(bsp, 52, qo, kv, 16, 4, 16, mode=mode, f8=f8, norm=True, max_gather_pages=100 if mode == "prefill" else 0)
    out, lse = (x.clone() for x in r())
    r.check(out, lse)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    o2, l2 = r(stream=st)
    torch.cuda.synchronize()
    assert torch.equal(out, o2) and torch.equal(lse, l2)
    o3, l3 = torch.empty_like(out), torch.empty_like(lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r(out=o3, lse=l3)
    for _ in range(2):
        o3.zero_()
        l3.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, o3) and torch.equal(lse, l3)
    assert torch.equal(r(return_lse=False), out)
    # a replay after another plan into the same workspace
    n = [1] * 3 if mode == "decode" else [100, 100, 21]
    r2 = Run(bsp, 53, n, [300, 600, 90], 16, 4, 16, mode=mode, f8=f8, norm=True)
    r.pa.plan(r2.b.kv_indptr, r2.b.last_page_len, qo_indptr=r2.b.qo_indptr)
    if r2.k.shape[0] <= r.k.shape[0]:
        for name in ("k", "v"):
            getattr(r, name).view(torch.uint8)[:r2.k.shape[0]] = getattr(r2, name).view(torch.uint8)
        for name, t in r.e.items():
            t[:r2.k.shape[0]] = r2.e[name]
        r.q.copy_(r2.q)
        r.lam_t.copy_(r2.lam_t)
        r.norm_t.copy_(r2.norm_t)
        r.idx[:r2.idx.numel()] = r2.idx
        graph.replay()
        torch.cuda.synchronize()
        r2.pa = r2.pa
        r2.check(o3, l3)


@pytest.mark.parametrize("mode", ["decode", "prefill"])
def test_results_on_another_stream_are_its_own(bsp, mode):
    from test_gpu_call_streams import freed_while_in_use
    qo = [1] * 300 if mode == "decode" else [300]
    r = Run(bsp, 54, qo, [33] * 300 if mode == "decode" else [300], 16, 4, 16, mode=mode)
    want = [t.clone() for t in r()]
    for shape, dtype in ((r.q.shape, torch.bfloat16), (r.q.shape[:2] + (2,), torch.float32)):
        got, kept = freed_while_in_use(shape, dtype, lambda s: r(stream=s))
        assert kept and all(torch.equal(a, b) for a, b in zip(got, want))


def test_no_queries(bsp):
    r = Run(bsp, 55, [0, 0], [40, 7], 16, 4, 16, mode="prefill")
    out, lse = r()
    assert out.shape == (0, 16, 128) and lse.shape == (0, 16, 2)


def test_refusals_of_the_binding(bsp):
    for kw in (dict(dtype=torch.float32), dict(head_dim=64)):
        with pytest.raises(ValueError):
            bsp.PagedAttention(**{**dict(mode="decode", num_qo_heads=8, num_kv_heads=2, head_dim=128, page_size=16, differential=True), **kw})
    r = Run(bsp, 56, [1, 1], [40, 7], 16, 4, 16)
    ok = dict(q=r.q, k_pages=r.k, v_pages=r.v, kv_indices=r.idx, lam=r.lam_t)
    for bad in (dict(q=r.q[:1]), dict(q=r.q.float()), dict(k_pages=r.k[:, :8]), dict(v_pages=r.v.float()), dict(kv_indices=r.idx[:1]),
                dict(lam=r.lam_t[:3]), dict(lam=r.lam_t.double()), dict(norm_weight=r.lam_t), dict(out=r.q[:, :3]), dict(lse=r.lam_t),
                dict(k_exp=torch.zeros(r.k.shape[0], 4, dtype=torch.int8, device="cuda")), dict(q=r.q.cpu())):
        with pytest.raises(ValueError):
            r.pa.run_differential(**{**ok, **bad})
    with pytest.raises(RuntimeError):
        r.pa.run(r.q, r.k, r.v, r.idx)
    with pytest.raises(RuntimeError):
        bsp.PagedAttention("decode", 8, 2, 128, 16).run_differential(**ok)
    with pytest.raises(bsp.BspError):  # nine heads, 18 maps per kv head
        Run(bsp, 57, [1], [40], 9, 1, 16)()


@pytest.mark.parametrize("mode", ["decode", "prefill"])
def test_weights_and_eviction_after_differential_attention(bsp, mode):
    """The serving loop over a differential cache: attention, weights |p1 - lam p2|, the choice, the move, and attention again."""
    qo = [1, 1, 1] if mode == "decode" else [64, 33, 5]
    r = Run(bsp, 58, qo, [700, 33, 300], 16, 4, 16, mode=mode, lam=0.7)
    b = r.b
    out, lse = r()
    t = dev(b.kv_indptr.astype(np.int32)), r.idx, dev(b.last_page_len.astype(np.int32))
    w = torch.full((r.k.shape[0], 4, 16), float("nan"), device="cuda")
    bsp.accumulate_weights(r.q, lse, r.k, w, *t, qo_indptr=dev(b.qo_indptr.astype(np.int32)), decay=0.0, lam=r.lam_t)
    want, size = ev.weights(b.q.double().numpy(), lse.double().cpu().numpy(), r.k64, np.zeros(w.shape), b.qo_indptr, b.kv_indptr,
                            b.kv_indices, b.last_page_len, 0.125, decay=0.0, lam=r.lam)
    got = w.double().cpu().numpy()
    used = size > 0
    # (the weights' own tests hold the tight bound: here that the run's LSE is the one that they take)
    assert (np.abs(got - want)[used] <= 2e-4 * size[used]).all()
    budget = torch.tensor([200, 50, 100], dtype=torch.int32, device="cuda")
    kept, new = bsp.select_tokens(w, *t, budget, 200, 4, 16)
    before = r.k.clone(), r.v.clone()
    bsp.compact_cache(kept, new, *t, r.k, r.v, weights=w)
    torch.cuda.synchronize()
    assert new.tolist() == [200, 33, 100]
    kk, n = kept.cpu().numpy(), new.cpu().numpy()
    for t0, t1 in zip(before, (r.k, r.v)):
        a = ev.compact(t0.view(torch.int16).cpu().numpy(), kk, n, b.kv_indptr, b.kv_indices, 16)
        assert np.array_equal(t1.view(torch.int16).cpu().numpy(), a)
    np_ = -(-n // 16)
    idx = np.concatenate([b.kv_indices[b.kv_indptr[i]:b.kv_indptr[i] + np_[i]] for i in range(3)]).astype(np.int32)
    one = Run(bsp, 59, [1, 1, 1], n.tolist(), 16, 4, 16, mode="decode", lam=0.7)
    one.k, one.v, one.idx = r.k, r.v, dev(idx)
    one.b.kv_indices[:] = idx
    one.k64, one.v64 = (x.double().cpu().numpy() for x in (r.k, r.v))
    one.check(*one())
