"""Measured cases of differential attention over the paged KV cache, and of the eviction of cached tokens by the
attention weight that they gathered.

Rows of q, k and v have 128 values. In differential attention a row of q and of k is two halves of 64, and a head's
output is the difference of the two softmax maps, applied to the whole rows of v:

    o = (softmax(scale q1 k1^T) - lam softmax(scale q2 k2^T)) v,    then, if asked for, o / rms(o) * norm weight * out_scale

Each cached token has a gathered weight per kv head, weights float32 [pages, kv heads, page_size]. Operators:

- diff_decode, diff_prefill: differential attention, one query per request, or several (causal)
- weights: after an attention run, the weight that each key got from the queries (a sum of softmax values over the queries
  and the query heads of a kv head) is added to its gathered weight times decay; a query's own key starts from zero
- select:  per request and kv head the tokens to keep: the first `sinks`, the last `recent`, then the heaviest
- compact: the kept tokens' rows move to the front of their request's pages, in order

Where ``own`` is false, run() computes them in elementary torch operations; where it is true, through the package.
"""
import math
import random

import numpy as np
import torch

own = False

D = 128  # values of a row


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one decoding request with a short cache: latency
        dict(name="diff_decode_1_short", op="diff_decode", batch=1, ps=16, hq=32, hk=8, lo=333, hi=333, new=1, f8=False,
             norm=True, window=0, cap=0.0, ls=1),
        # a decode batch of 64 requests, up to 8192 tokens each, 16-token pages, normalised heads
        dict(name="diff_decode_64", op="diff_decode", batch=64, ps=16, hq=32, hk=8, lo=512, hi=8192, new=1, f8=False,
             norm=True, window=0, cap=0.0, ls=2),
        # a short prompt behind a short cache, no norm
        dict(name="diff_prefill_small", op="diff_prefill", batch=2, ps=16, hq=32, hk=8, lo=0, hi=150, new=70, f8=False,
             norm=False, window=0, cap=0.0, ls=3),
        # 16 ragged prompts, nothing cached before
        dict(name="diff_prefill_ragged", op="diff_prefill", batch=16, ps=16, hq=32, hk=8, lo=0, hi=0, new=2048, f8=False,
             norm=True, window=0, cap=0.0, ls=4),
        # the step of 64 decoding requests: each key's weight grows by what the new token's heads gave it
        dict(name="weights_decode_64", op="weights", batch=64, ps=16, hq=32, hk=8, lo=512, hi=8192, new=1, kind="bf16",
             decay=1.0, diff=False, window=0, cap=0.0, ls=5),
        # the same over an 8-bit cache, older weights fading, 64 query heads over 8
        dict(name="weights_decode_8bit", op="weights", batch=32, ps=16, hq=64, hk=8, lo=4096, hi=4096, new=1, kind="e4m3",
             decay=0.97, diff=False, window=0, cap=0.0, ls=6),
        # whole prompts: every query's weights
        dict(name="weights_prompts", op="weights", batch=2, ps=16, hq=32, hk=8, lo=6000, hi=8192, new=1 << 30, kind="bf16",
             decay=0.0, diff=False, window=0, cap=0.0, ls=7),
        # the tokens to keep of 64 grown requests, half of each cache
        dict(name="select_64", op="select", batch=64, ps=16, hk=8, lo=2000, hi=8192, keep=2048, sinks=4, recent=64,
             ties=False, ls=8),
        # one long prompt down to 4096 tokens
        dict(name="select_long", op="select", batch=1, ps=16, hk=8, lo=131072, hi=131072, keep=4096, sinks=4, recent=512,
             ties=False, ls=9),
        # a small step: four requests, a few hundred tokens, latency
        dict(name="compact_4_short", op="compact", batch=4, ps=16, hk=8, lo=300, hi=500, keep=256, sinks=4, recent=32,
             kind="bf16", ls=10),
        # a batch that grew by 128 tokens since the last eviction
        dict(name="compact_64", op="compact", batch=64, ps=16, hk=8, lo=2176, hi=2176, keep=2048, sinks=4, recent=64,
             kind="bf16", ls=11),
        # long prompts in an 8-bit cache down to 4096 tokens each
        dict(name="compact_prompts_8bit", op="compact", batch=4, ps=16, hk=8, lo=16000, hi=32768, keep=4096, sinks=4,
             recent=512, kind="e4m3", ls=12),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["diff_decode", "diff_decode", "diff_prefill", "diff_prefill", "weights", "weights", "select", "compact"])
    ls = rng.randrange(1 << 20)
    ps = rng.choice([1, 5, 8, 12, 16, 32, 64, 128])
    if op in ("diff_decode", "diff_prefill"):
        decode = op == "diff_decode"
        hq, hk = rng.choice([(32, 8), (16, 2), (8, 8), (16, 4), (8, 1)] + ([(24, 8), (15, 5)] if decode else [(32, 2)]))
        batch = _log_int(rng, 1, 64 if decode else 12)
        hi = _log_int(rng, 8, max(16, min(32768, 1600000 // (batch * hk)))) if decode else _log_int(rng, 1, 4096 // batch)
        return dict(op=op, batch=batch, ps=ps, hq=hq, hk=hk, lo=max(1, hi // 8) if decode else 0, hi=hi,
                    new=1 if decode else _log_int(rng, 2, 3600 // batch), f8=rng.random() < 0.3, norm=rng.random() < 0.6,
                    window=rng.choice([0, 0, 0, max(1, hi // 3)]), cap=rng.choice([0.0, 0.0, 30.0]), ls=ls)
    if op == "weights":
        kind = rng.choice(["bf16", "bf16", "bf16", "e4m3", "f32"])
        hq, hk = rng.choice([(32, 8), (64, 8), (16, 2), (8, 8), (12, 4), (5, 1)])
        diff = kind != "f32" and hq // hk <= 8 and rng.random() < 0.3
        batch = _log_int(rng, 1, 64)
        new = rng.choice([1, 1, _log_int(rng, 2, 256), 1 << 30] if kind == "bf16" else [1, 1, _log_int(rng, 2, 32)])
        most = 1600000 // (batch * hk) // (2 if kind == "f32" else 1)
        if new > 1:  # (query, key) pairs of all heads
            most = min(most, int(math.sqrt(1e9 / (batch * hq))) if new > 256 else int(1e9 / (batch * hq * new)), 16384)
        hi = _log_int(rng, 4, max(8, min(32768, most)))
        return dict(op=op, batch=batch, ps=ps, hq=hq, hk=hk, lo=max(1, hi // 4), hi=hi, new=new, kind=kind,
                    decay=rng.choice([1.0, 1.0, 0.95, 0.0]), diff=diff, window=rng.choice([0, 0, 0, max(1, hi // 3)]),
                    cap=rng.choice([0.0, 0.0, 30.0]), ls=ls)
    hk = rng.choice([1, 2, 5, 8, 8])
    batch = _log_int(rng, 1, 64)
    hi = _log_int(rng, 2, max(4, min(131072, (4000000 if op == "select" else 1000000) // (batch * hk))))
    sinks, recent = rng.choice([0, 1, 4]), rng.choice([0, 1, 32, 300])
    keep = max(1, sinks + recent, int(hi * rng.uniform(0.02, 1.1)))
    c = dict(op=op, batch=batch, ps=ps, hk=hk, lo=rng.choice([0, hi // 2]), hi=hi, keep=keep, sinks=sinks, recent=recent)
    if op == "select":
        return dict(c, ties=rng.random() < 0.4, ls=ls)
    return dict(c, kind=rng.choice(["bf16", "bf16", "e4m3", "f32"]), ls=ls)


def _lens(case):
    """(tokens in the cache, queries or tokens to keep) of each request: fixed by the case."""
    r = np.random.default_rng(case["ls"])
    B, lo, hi = case["batch"], case["lo"], case["hi"]
    lens = r.integers(lo, hi + 1, size=B).astype(np.int64)
    if case["op"] in ("select", "compact"):
        keep = r.integers((case["keep"] + 1) // 2, case["keep"] + 1, size=B) if lo != hi else np.full(B, case["keep"])
        return lens, keep.astype(np.int64)
    n = case["new"]
    if case["op"] == "diff_prefill":
        new = r.integers((n + 1) // 2, n + 1, size=B).astype(np.int64)
        return lens + new, new
    return lens, np.minimum(lens, n)


def _pages(lens, ps):
    return (lens + ps - 1) // ps


def _visible(kv, new, window):
    """Visible (query, key) pairs per head: query i of a request sees keys up to kv - new + i, within the window."""
    first = kv - new + 1  # keys that the first query sees
    if not window:
        return int((new * first + new * (new - 1) // 2).sum())
    short = np.clip(window + 1 - first, 0, new)  # queries that see fewer keys than the window has
    return int((short * first + short * (short - 1) // 2 + (new - short) * (window + 1)).sum())


def work(case):
    kv, new = _lens(case)
    ps, hk, op = case["ps"], case["hk"], case["op"]
    tokens, pages = int(kv.sum()), int(_pages(kv, ps).sum())
    if op == "select":
        return {"bytes": 4 * hk * tokens + 4 * pages + 4 * hk * case["batch"] * int(new.max()) + 4 * 4 * case["batch"], "flops": 0}
    if op == "compact":
        kept = int(np.where(kv > new, new, 0).sum())  # rows that move: nearly all kept ones of the longer requests
        row = 2 * D * {"bf16": 2, "f32": 4, "e4m3": 1}[case["kind"]] + 4
        return {"bytes": hk * kept * (2 * row + 4) + 4 * pages, "flops": 0}
    n, w, hq = int(new.sum()), case["window"], case["hq"]
    pairs = _visible(kv, new, w)
    read = int((np.minimum(kv, w + new) if w else kv).sum())
    if op == "weights":
        elem = {"bf16": 2, "f32": 4, "e4m3": 1}[case["kind"]]
        maps = 2 if case["diff"] else 1
        b = read * hk * D * elem + tokens * hk * (4 if case["decay"] == 0 else 8) + n * hq * (D * (4 if elem == 4 else 2) + 4 * maps)
        return {"bytes": b + 4 * pages, "flops": 2 * D * hq * pairs}
    b = read * hk * D * 2 * (1 if case["f8"] else 2) + n * hq * (D * 4 + 8) + 4 * pages
    return {"bytes": b, "flops": (2 * D + 2 * 2 * D) * hq * pairs}  # two maps: halves of 64, then whole rows of v


# ---------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _indptr(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)


def _pow2(e):
    """2^e in 32 bits, exactly, for whole e in [-126, 127] (below: 2^-126)."""
    return ((e.int().clamp(-126, 127) + 127) << 23).view(torch.float32)


def _take(codes, at):
    """codes[at] of an e4m3 array, as 32-bit values (indexed as bytes)."""
    return codes.view(torch.uint8)[at].view(torch.float8_e4m3fn).float()


def _pool(g, kind, num_pages, ps, hk):
    """A filled pool [pages, page_size, kv heads, D] and its exponents [pages, kv heads] (e4m3) or None."""
    if kind != "e4m3":
        x = torch.randn((num_pages, ps, hk, D), generator=g, device="cuda")
        return x.to(torch.float32 if kind == "f32" else torch.bfloat16), None
    e = torch.randint(-8, -5, (num_pages, hk), generator=g, device="cuda", dtype=torch.int32)
    x = torch.randn((num_pages, ps, hk, D), generator=g, device="cuda")
    return (x * 100.0).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn), e.to(torch.int8)


def _heavy(g, shape):
    """Gathered weights: heavy-tailed, a few tokens have most of them."""
    return torch.exp(torch.randn(shape, generator=g, device="cuda") * 2.0)


def prepare(case, seed):
    g = _gen(seed)
    kv, new = _lens(case)
    ps, hk, B, op = case["ps"], case["hk"], case["batch"], case["op"]
    pages = _pages(kv, ps)
    num_pages = int(pages.sum()) + 5
    perm = torch.randperm(num_pages, generator=g, device="cuda").to(torch.int32)
    last = np.where(pages > 0, (kv - 1) % ps + 1, 0)
    # the page table in CSR form, on the device (as bsp.build_page_tables leaves it)
    s = dict(case=case, kv_indptr=_i32(_indptr(pages)), kv_indices=perm[:int(pages.sum())].contiguous(), last=_i32(last),
             most_pages=int(pages.max()))
    if op in ("select", "compact"):
        s["most"] = int(new.max())
        s["budget"] = _i32(new)
        w = _heavy(g, (num_pages, hk, ps))
        if case.get("ties"):
            w = torch.floor(w)  # many equal weights, many zeros
        s["weights"] = w
        if op == "compact":  # what to keep is decided: sorted positions, behind the last -1
            T = int(kv.max())
            x = torch.rand((B, hk, max(T, s["most"])), generator=g, device="cuda")
            t = torch.arange(x.shape[2], device="cuda")
            L = torch.from_numpy(kv).cuda()[:, None, None]
            x = torch.where((t < case["sinks"]) | (t >= L - case["recent"]), 2.0, x)
            x = torch.where(t < L, x, -1.0)
            n = torch.from_numpy(np.minimum(kv, new)).cuda()
            place = torch.arange(s["most"], device="cuda")
            top = torch.topk(x, s["most"], dim=2).indices
            top = torch.where(place < n[:, None, None], top, 1 << 30).sort(dim=2).values
            s["kept"] = torch.where(place < n[:, None, None], top, -1).to(torch.int32).contiguous()
            s["new_lens"] = n.to(torch.int32)
            s["k"], s["k_exp"] = _pool(g, case["kind"], num_pages, ps, hk)
            s["v"], s["v_exp"] = _pool(g, case["kind"], num_pages, ps, hk)
        return s
    n, hq = int(new.sum()), case["hq"]
    s["qo_indptr"] = _i32(_indptr(new))
    s["most_new"] = int(new.max())
    kind = case["kind"] if op == "weights" else "e4m3" if case["f8"] else "bf16"
    two = op != "weights" or case["diff"]
    s["scale"] = 1.0 / math.sqrt(D // 2 if two else D)
    q = torch.randn((n, hq, D), generator=g, device="cuda")
    s["q"] = q.to(torch.float32 if kind == "f32" else torch.bfloat16)
    s["k"], s["k_exp"] = _pool(g, kind, num_pages, ps, hk)
    if two:  # one factor per head, around the 0.8 that training starts from
        s["lam"] = 0.8 + 0.1 * torch.randn((hq,), generator=g, device="cuda")
    if op == "weights":
        s["weights"] = _heavy(g, (num_pages, hk, ps))

        def normalisers(maps):
            """log-sum-exp of every query's scores, as the attention run before left it."""
            lse = torch.empty((n, hq, maps), device="cuda")
            qp, kp, gr, d = _indptr(new), _indptr(pages), hq // hk, D // maps
            for b in range(B):
                ids = s["kv_indices"][int(kp[b]):int(kp[b + 1])].long()
                N, L = int(new[b]), int(kv[b])
                own_pos = torch.arange(L - N, L, device="cuda")[None, :, None]
                t = torch.arange(L, device="cuda")
                gone = t > own_pos
                if case["window"] > 0:
                    gone = gone | (t < own_pos - case["window"])
                for h in range(hk):
                    if kind == "e4m3":
                        k = s["k"].view(torch.uint8)[ids, :, h].view(torch.float8_e4m3fn).float()
                        k = k * _pow2(s["k_exp"][ids, h])[:, None, None]
                    else:
                        k = s["k"][ids, :, h].float()
                    k = k.reshape(-1, D)[:L]
                    for m in range(maps):
                        qh = s["q"][int(qp[b]):int(qp[b + 1]), h * gr:(h + 1) * gr, m * d:(m + 1) * d].float()
                        x = torch.matmul(qh.transpose(0, 1), k[:, m * d:(m + 1) * d].T).mul_(s["scale"])
                        if case["cap"] > 0:
                            x = torch.tanh(x / case["cap"]) * case["cap"]
                        x.masked_fill_(gone, -math.inf)
                        lse[int(qp[b]):int(qp[b + 1]), h * gr:(h + 1) * gr, m] = torch.logsumexp(x, dim=2).T
            return lse

        lse = normalisers(2 if two else 1)
        s["lse"] = lse.contiguous() if two else lse[:, :, 0].contiguous()
        return s
    s["v"], s["v_exp"] = _pool(g, kind, num_pages, ps, hk)
    s["norm"] = 1.0 + 0.1 * torch.randn((D,), generator=g, device="cuda") if case["norm"] else None
    s["out_scale"] = 0.2 if case["norm"] else 1.0
    if own:
        import block_sparse_paged_gb300 as bsp
        decode = op == "diff_decode"
        pa = bsp.PagedAttention("decode" if decode else "prefill", hq, hk, D, ps, causal=not decode, dtype=torch.bfloat16,
                                max_batch=B, max_qo_tokens=n, window_left=case["window"], logits_soft_cap=case["cap"],
                                differential=True)
        pa.plan(_indptr(pages), last, qo_indptr=None if decode else _indptr(new))
        s["attention"] = pa
    return s


# ---------------------------------------------------------------- plain forms
def _table(s):
    """Padded page ids [B, most pages], whether each is there, and the tokens of each request."""
    ps = s["case"]["ps"]
    kvp = s["kv_indptr"].long()
    count = kvp[1:] - kvp[:-1]
    j = torch.arange(s["most_pages"], device=kvp.device)
    if s["kv_indices"].numel() == 0:
        pages = torch.zeros((count.numel(), s["most_pages"]), dtype=torch.int64, device=kvp.device)
    else:
        pages = s["kv_indices"].long()[(kvp[:-1, None] + j).clamp(max=s["kv_indices"].numel() - 1)]
    return pages, j < count[:, None], torch.where(count > 0, (count - 1) * ps + s["last"].long(), 0)


def _queries(s, lens):
    """Rows of q [B, most queries], whether each is there, and its position among its request's keys."""
    qop = s["qo_indptr"].long()
    nq = qop[1:] - qop[:-1]
    i = torch.arange(s["most_new"], device=qop.device)
    row = (qop[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    return row, i < nq[:, None], (lens - nq)[:, None] + i


def _keys(codes, exps, pages):
    """Padded rows [B, T, kv heads, D] in 32 bits."""
    x = codes[pages].float() if exps is None else _take(codes, pages) * _pow2(exps[pages])[:, :, None, :, None]
    return x.flatten(1, 2)


def _scores(s, maps, pages, lens, row, pos):
    """Scaled, capped and masked scores [B, kv heads, maps, group, Q, T] and the mask [B, Q, T]."""
    c = s["case"]
    hk, gr, d = c["hk"], c["hq"] // c["hk"], D // maps
    B, Q = row.shape
    k = _keys(s["k"], s["k_exp"], pages).unflatten(3, (maps, d)).permute(0, 2, 3, 4, 1)
    q = s["q"][row].float().view(B, Q, hk, gr, maps, d).permute(0, 2, 4, 3, 1, 5).reshape(B, hk, maps, gr * Q, d)
    x = torch.matmul(q, k).mul_(s["scale"]).view(B, hk, maps, gr, Q, -1)
    if c["cap"] > 0:
        x = torch.tanh(x / c["cap"]).mul_(c["cap"])
    t = torch.arange(x.shape[-1], device=x.device)
    see = (t <= pos[:, :, None]) & (t < lens[:, None, None])
    if c["window"] > 0:
        see = see & (t >= pos[:, :, None] - c["window"])
    return x.masked_fill_(~see[:, None, None, None], -math.inf), see


def _plain_diff(s):
    c = s["case"]
    hq, hk = c["hq"], c["hk"]
    gr = hq // hk
    pages, _, lens = _table(s)
    row, live, pos = _queries(s, lens)
    B, Q = row.shape
    x, _ = _scores(s, 2, pages, lens, row, pos)
    T = x.shape[-1]
    m = x.amax(dim=-1, keepdim=True)
    m = torch.where(torch.isinf(m), 0.0, m)
    x = x.sub_(m).exp_()
    l = x.sum(dim=-1, keepdim=True)
    v = _keys(s["v"], s["v_exp"], pages)
    seen = torch.arange(T, device=v.device) < lens[:, None]
    v = torch.where(seen[:, :, None, None], v, 0.0).permute(0, 2, 1, 3)
    o = torch.matmul(x.view(B, hk, 2 * gr * Q, T), v).view(B, hk, 2, gr, Q, D) / l
    o = o[:, :, 0] - s["lam"].view(hk, gr, 1, 1) * o[:, :, 1]
    if s["norm"] is not None:
        o = o * torch.rsqrt((o * o).mean(dim=-1, keepdim=True) + 1e-5) * s["norm"]
    o = o * s["out_scale"]
    lse = (m + torch.log(l)).squeeze(-1)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, Q, hq, D)[live]
    lse = lse.permute(0, 4, 1, 3, 2).reshape(B, Q, hq, 2)[live]
    return {"o": o.to(torch.bfloat16), "lse": lse}


def _plain_weights(s):
    c = s["case"]
    hk, ps, maps = c["hk"], c["ps"], 2 if c["diff"] else 1
    gr = c["hq"] // hk
    pages, there, lens = _table(s)
    row, live, pos = _queries(s, lens)
    B, Q = row.shape
    x, _ = _scores(s, maps, pages, lens, row, pos)
    lse = s["lse"][row].view(B, Q, hk, gr, maps).permute(0, 2, 4, 3, 1)[..., None]
    x = x.sub_(lse).exp_()
    if maps == 2:
        x = (x[:, :, 0] - s["lam"].view(hk, gr, 1, 1) * x[:, :, 1]).abs_()
    else:
        x = x[:, :, 0]
    x = (x * live[:, None, None, :, None]).sum(dim=(2, 3))  # [B, kv heads, T]
    t = torch.arange(x.shape[-1], device=x.device)
    fresh = t >= (lens - live.sum(dim=1))[:, None]
    old = s["weights"][pages].permute(0, 2, 1, 3).reshape(B, hk, -1)
    base = torch.where(fresh[:, None], 0.0, old * c["decay"]) if c["decay"] else torch.zeros_like(old)
    w = torch.where((t < lens[:, None])[:, None], base + x, old)
    w = w.view(B, hk, -1, ps).permute(0, 2, 1, 3)
    s["weights"][pages[there]] = w[there]
    return {"weights": s["weights"]}


def _plain_select(s):
    c = s["case"]
    pages, _, lens = _table(s)
    B, hk, K = pages.shape[0], c["hk"], s["most"]
    w = s["weights"][pages].permute(0, 2, 1, 3).reshape(B, hk, -1)
    T = max(w.shape[2], K)
    w = torch.nn.functional.pad(w, (0, T - w.shape[2]))
    t = torch.arange(T, device=w.device)
    L = lens[:, None, None]
    w = torch.where((t < c["sinks"]) | (t >= L - c["recent"]), math.inf, w)
    w = torch.where(t < L, w, -math.inf)
    n = torch.minimum(lens, s["budget"].long())
    order = torch.sort(w, dim=2, descending=True, stable=True).indices[:, :, :K]
    place = torch.arange(K, device=w.device)
    inside = place < n[:, None, None]
    kept = torch.where(inside, order, 1 << 30).sort(dim=2).values
    return {"kept": torch.where(inside, kept, -1).int(), "new_lens": n.int()}


def _plain_compact(s):
    c = s["case"]
    ps, hk = c["ps"], c["hk"]
    pages, _, _ = _table(s)
    K = s["most"]
    place = torch.arange(K, device=pages.device)
    b, h, j = torch.nonzero(place < s["new_lens"][:, None, None].expand(-1, hk, -1), as_tuple=True)
    i = s["kept"][b, h, j].long()
    sp, dp = pages[b, i // ps], pages[b, j // ps]
    si, di = i % ps, j % ps
    s["weights"][dp, h, di] = s["weights"][sp, h, si]
    if c["kind"] != "e4m3":
        s["k"][dp, di, h] = s["k"][sp, si, h]
        s["v"][dp, di, h] = s["v"][sp, si, h]
        return {"k": s["k"], "v": s["v"], "weights": s["weights"]}
    at = dp * hk + h
    _move_codes(s["k"], s["k_exp"], sp, si, dp, di, h, at)
    _move_codes(s["v"], s["v_exp"], sp, si, dp, di, h, at)
    return {"k": s["k"], "v": s["v"], "k_exp": s["k_exp"], "v_exp": s["v_exp"], "weights": s["weights"]}


def _move_codes(codes, exps, sp, si, dp, di, h, at):
    """Rows of codes to their new places, each page's exponent the largest of those that its rows had."""
    had = exps[sp, h].int()
    e = torch.full((exps.numel(),), -128, dtype=torch.int32, device=exps.device).scatter_reduce(0, at, had, "amax")
    x = _take(codes, (sp, si, h)) * _pow2(had - e[at])[:, None]
    codes.view(torch.uint8)[dp, di, h] = x.to(torch.float8_e4m3fn).view(torch.uint8)
    exps.view(-1)[at] = e[at].to(torch.int8)


# ---------------------------------------------------------------- one pass
def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if own:
        import block_sparse_paged_gb300 as bsp
        table = (s["kv_indptr"], s["kv_indices"], s["last"])
        if op == "weights":
            bsp.accumulate_weights(s["q"], s["lse"], s["k"], s["weights"], *table, qo_indptr=s["qo_indptr"],
                                   sm_scale=s["scale"], decay=c["decay"], k_exp=s["k_exp"], lam=s.get("lam"),
                                   window_left=c["window"], logits_soft_cap=c["cap"])
            return {"weights": s["weights"]}
        if op == "select":
            kept, new_lens = bsp.select_tokens(s["weights"], *table, s["budget"], s["most"], sinks=c["sinks"],
                                               recent=c["recent"])
            return {"kept": kept, "new_lens": new_lens}
        if op == "compact":
            bsp.compact_cache(s["kept"], s["new_lens"], *table, s["k"], s["v"], weights=s["weights"], k_exp=s["k_exp"],
                              v_exp=s["v_exp"])
            out = {"k": s["k"], "v": s["v"], "weights": s["weights"]}
            return out if s["k_exp"] is None else dict(out, k_exp=s["k_exp"], v_exp=s["v_exp"])
        o, lse = s["attention"].run_differential(s["q"], s["k"], s["v"], s["kv_indices"], s["lam"], sm_scale=s["scale"],
                                                 norm_weight=s["norm"], norm_eps=1e-5, out_scale=s["out_scale"],
                                                 k_exp=s["k_exp"], v_exp=s["v_exp"])
        return {"o": o, "lse": lse}
    if op == "weights":
        return _plain_weights(s)
    if op == "select":
        return _plain_select(s)
    if op == "compact":
        return _plain_compact(s)
    return _plain_diff(s)


# ---------------------------------------------------------------- 64 bits
def _two_to(e):
    """2^e in 64 bits from its bits, for whole e in [-1022, 1023]."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _e4m3_64(y):
    """Nearest e4m3 value (ties to even) of float64 y with |y| <= 448: three bits after the leading one, spacing at
    least 2^-9."""
    _, ex = torch.frexp(y.abs())  # |y| = m 2^ex, m in [0.5, 1)
    step = _two_to((ex - 4).clamp(min=-9))
    return torch.round(y / step) * step  # torch.round: half to even


def _rows64(codes, exps, ids, h, L):
    """Rows of one request and kv head in 64 bits."""
    if exps is None:
        return codes[ids, :, h].double().reshape(-1, D)[:L]
    x = codes.view(torch.uint8)[ids, :, h].view(torch.float8_e4m3fn).double()
    return (x * _two_to(exps[ids, h])[:, None, None]).reshape(-1, D)[:L]


def _each_head(s):
    """(request, first query row, behind the last, page ids, tokens, masked (query, key) pairs, kv head) one by one."""
    c = s["case"]
    kp, qp, last = s["kv_indptr"].tolist(), s["qo_indptr"].tolist(), s["last"].tolist()
    for b in range(c["batch"]):
        ids = s["kv_indices"][kp[b]:kp[b + 1]].long()
        L = max(0, (len(ids) - 1) * c["ps"] + last[b])
        at = torch.arange(L - qp[b + 1] + qp[b], L, device="cuda")[:, None]
        t = torch.arange(L, device="cuda")
        gone = t > at
        if c["window"] > 0:
            gone = gone | (t + c["window"] < at)
        for h in range(c["hk"]):
            yield b, qp[b], qp[b + 1], ids, L, gone, h


def _score64(s, q, k, gone):
    z = (q.double() @ k.T) * s["scale"]
    if s["case"]["cap"] > 0:
        z = s["case"]["cap"] * torch.tanh(z / s["case"]["cap"])
    return z.masked_fill_(gone, -math.inf)


def exact(case, seed):
    global own
    op = case["op"]
    if op == "select":
        return None  # whole numbers
    keep, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = keep
    ps, hk = case["ps"], case["hk"]
    if op == "compact":
        if case["kind"] != "e4m3":
            return None  # values that move as they are
        kp, kept, lens = s["kv_indptr"].tolist(), s["kept"].cpu().numpy(), s["new_lens"].tolist()
        ids = s["kv_indices"].cpu().numpy()
        out = {"weights": None, "k_exp": None, "v_exp": None}
        for name in ("k", "v"):
            was = s[name].double()
            had = s[name + "_exp"].cpu().numpy().astype(np.int64)
            now = was.clone()
            for b in range(case["batch"]):
                row = ids[kp[b]:kp[b + 1]]
                for h in range(hk if lens[b] else 0):
                    src = kept[b, h, :lens[b]].astype(np.int64)
                    e = had[row[src // ps], h]
                    starts = np.arange(0, lens[b], ps)
                    e_new = np.repeat(np.maximum.reduceat(e, starts), ps)[:lens[b]]
                    x = was[torch.from_numpy(row[src // ps]).cuda().long(), torch.from_numpy(src % ps).cuda(), h]
                    j = np.arange(lens[b])
                    x = _e4m3_64(x * _two_to(torch.from_numpy(e - e_new).cuda())[:, None])
                    now[torch.from_numpy(row[j // ps]).cuda().long(), torch.from_numpy(j % ps).cuda(), h] = x
            out[name] = now
        return out
    gr = case["hq"] // hk
    if op == "weights":
        w, maps = s["weights"].double(), 2 if case["diff"] else 1
        d, lse = D // maps, s["lse"].double().view(-1, case["hq"], maps)
        for b, q0, q1, ids, L, gone, h in _each_head(s):
            if not L:
                continue
            k = _rows64(s["k"], s["k_exp"], ids, h, L)
            got = torch.zeros(L, dtype=torch.float64, device="cuda")
            for r in range(gr * h, gr * h + gr):
                p = [torch.exp(_score64(s, s["q"][q0:q1, r, m * d:(m + 1) * d], k[:, m * d:(m + 1) * d], gone)
                               - lse[q0:q1, r, m, None]) for m in range(maps)]
                got += (p[0] if maps == 1 else (p[0] - s["lam"][r].double() * p[1]).abs()).sum(dim=0)
            t = torch.arange(L, device="cuda")
            page, place = ids[t // ps], t % ps
            old = w[page, h, place] * case["decay"]
            old[L - (q1 - q0):] = 0.0
            w[page, h, place] = old + got
        return {"weights": w}
    n = s["q"].shape[0]
    o = torch.zeros((n, case["hq"], D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((n, case["hq"], 2), dtype=torch.float64, device="cuda")
    for b, q0, q1, ids, L, gone, h in _each_head(s):
        k, v = _rows64(s["k"], s["k_exp"], ids, h, L), _rows64(s["v"], s["v_exp"], ids, h, L)
        for r in range(gr * h, gr * h + gr):
            a = []
            for m in range(2):
                z = _score64(s, s["q"][q0:q1, r, m * 64:m * 64 + 64], k[:, m * 64:m * 64 + 64], gone)
                lse[q0:q1, r, m] = torch.logsumexp(z, dim=1)
                a.append(torch.exp(z - lse[q0:q1, r, m][:, None]))
            y = (a[0] - s["lam"][r].double() * a[1]) @ v
            if s["norm"] is not None:
                y = y / torch.sqrt((y * y).mean(dim=1, keepdim=True) + 1e-5) * s["norm"].double()
            o[q0:q1, r] = y * s["out_scale"]
    return {"o": o, "lse": lse}


if __name__ == "__main__":
    rng_ = random.Random(1)
    for case_ in listed() + [draw(rng_) for _ in range(12)]:
        print(case_, work(case_))
