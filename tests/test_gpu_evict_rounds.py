"""Rounds of serving with eviction: tokens appended to a cache that was compacted, attention over it, gathered weights, the
choice and the move, each held against its plain form on what the round before left on the GPU. (The bounds are those of
the calls' own tests.)"""
import numpy as np
import pytest
import torch

import oracle
import workloads
from gpu_helpers import lib
from oracle import evict as ev
from oracle import kv_cache as kc
from test_gpu_evict import F8, bound, dev, serving_step
from test_gpu_fp8_block import check, reference

pytestmark = pytest.mark.gpu
PS, HQ, HK, P = 16, 16, 4, 90


@pytest.fixture(scope="module")
def bsp():
    return lib()


def test_attention_over_a_compacted_8bit_cache(bsp):
    """The codes that the move rescaled are what attention reads next: no tolerance but attention's own."""
    s, step, _, b = serving_step(bsp, "e4m3")
    step()
    torch.cuda.synchronize()
    new = s["new"].cpu().numpy()
    pages = -(-new // PS)
    indptr = np.concatenate([[0], np.cumsum(pages)]).astype(np.int32)
    indices = np.concatenate([b.kv_indices[b.kv_indptr[i]:b.kv_indptr[i] + pages[i]] for i in range(4)]).astype(np.int32)
    last = ((new - 1) % PS + 1).astype(np.int32)
    c8 = [s[n].view(torch.uint8).cpu().numpy() if n in "kv" else s[n].cpu().numpy() for n in ("k", "ke", "v", "ve")]
    after = workloads.PagedBatch("after", "bf16", HQ, HK, 128, PS, False, 128 ** -0.5, b.qo_indptr, indptr, indices, last, b.q,
                                 torch.zeros(1), torch.zeros(1))
    pa = bsp.PagedAttention("decode", HQ, HK, 128, PS, max_batch=4)
    pa.plan(indptr, last)
    out, lse = pa.run(s["q"], s["k"], s["v"], dev(indices), k_exp=s["ke"], v_exp=s["ve"])
    torch.cuda.synchronize()
    assert pa.check_device_error() == 0
    check(out, lse, reference(after, c8), 2.0 ** -11, after)


@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "e4m3"])
def test_rounds(bsp, f8):
    rng = np.random.default_rng(91)
    B, width, scale = 4, 40, 128 ** -0.5
    if f8:
        k, v = (torch.zeros(P, PS, HK, 128, dtype=torch.uint8, device="cuda").view(F8) for _ in range(2))
        exps = dict(k_exp=torch.zeros(P, HK, dtype=torch.int8, device="cuda"), v_exp=torch.zeros(P, HK, dtype=torch.int8, device="cuda"))
    else:
        k, v = (torch.zeros(P, PS, HK, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        exps = {}
    w = torch.full((P, HK, PS), float("nan"), device="cuda")  # (what free slots hold says nothing)
    table, pool = torch.full((B, width), -1, dtype=torch.int32, device="cuda"), rng.permutation(P).astype(np.int32)
    lens = np.zeros(B, np.int64)

    def raw(t):
        return t.view(torch.uint8 if f8 else torch.int16).cpu().numpy()

    def cache():
        """float64 K and V."""
        if f8:
            return [kc.values(raw(t), e.cpu().numpy()) for t, e in zip((k, v), exps.values())]
        return [t.double().cpu().numpy() for t in (k, v)]
    # prompts, single tokens, a chunk for some, single tokens again
    for new, budget in [([70, 1, 33, 200], [40, 9, 33, 100]), ([1] * 4, [41, 9, 20, 90]), ([20, 0, 5, 17], [50, 9, 24, 64]),
                        ([1] * 4, [17, 10, 1, 33])]:
        new, n = np.array(new), int(np.sum(new))
        # the table, and the new tokens' rows into the cache
        free = torch.zeros(P, dtype=torch.int32, device="cuda")
        free[:len(pool)] = dev(pool)
        t = bsp.build_page_tables(dev(lens.astype(np.int32)), dev(new.astype(np.int32)), free, dev(np.array([len(pool)], np.int32)), table, PS,
                                  B * width, n)
        x = [torch.from_numpy(rng.standard_normal((n, HK, 128)) * np.exp2(rng.uniform(-3, 3, (n, 1, 1)))).bfloat16() for _ in range(2)]
        slots = t.slot_map.cpu().numpy()
        if f8:
            before = [(raw(c), e.cpu().numpy()) for c, e in zip((k, v), exps.values())]
            bsp.append_kv(x[0].cuda(), x[1].cuda(), t.slot_map, k, v, **exps)
            for c, e, was, xs in zip((k, v), exps.values(), before, x):
                want, we = kc.append(xs.double().numpy(), slots, *was)
                assert np.array_equal(raw(c), want) and np.array_equal(e.cpu().numpy(), we)
        else:
            for c, xs in zip((k, v), x):
                c.view(P * PS, HK, 128)[t.slot_map] = xs.cuda()
        pool = pool[int(t.counts[2]):]
        assert int(t.counts[3]) == 0
        lens = lens + new
        pages = int(t.counts[0])
        decode = (new == 1).all()
        q = torch.from_numpy(rng.standard_normal((n, HQ, 128))).bfloat16()
        b = workloads.PagedBatch("round", "bf16", HQ, HK, 128, PS, not decode, scale, t.qo_indptr.cpu().numpy(), t.kv_indptr.cpu().numpy(),
                                 t.kv_indices.cpu().numpy()[:pages], t.last_page_len.cpu().numpy(), q, torch.zeros(1), torch.zeros(1))
        assert np.array_equal(b.kv_lens, lens)
        # attention
        pa = bsp.PagedAttention("decode" if decode else "prefill", HQ, HK, 128, PS, not decode, max_batch=B, max_qo_tokens=n)
        pa.plan(b.kv_indptr, b.last_page_len, qo_indptr=None if decode else b.qo_indptr)
        out, lse = pa.run(q.cuda(), k, v, t.kv_indices, **exps)
        torch.cuda.synchronize()
        assert pa.check_device_error() == 0
        kv64 = cache()
        if f8:
            check(out, lse, reference(b, [raw(k), exps["k_exp"].cpu().numpy(), raw(v), exps["v_exp"].cpu().numpy()]),
                  2.0 ** -11 if decode else 2.0 ** -8, b)
        else:
            # (rows of up to 8 times the unit normal's size: each weight is rounded to bf16, 2^-8 of itself, so that an output
            # is off by 2^-8 of A = sum p |v|, beside the scores' errors and its own rounding, as over the 8-bit cache)
            O, L = oracle.attention_of(b, k=kv64[0], v=kv64[1])
            A, _ = oracle.attention_of(b, k=kv64[0], v=np.abs(kv64[1]))
            qk = scale * np.sqrt((b.q.float().numpy() ** 2).sum(-1)).max() * np.sqrt((kv64[0] ** 2).sum(-1)).max()
            check(out, lse, (O, L, A, qk), 2.0 ** -8, b)
        # weights: the new tokens' from zero
        was = w.cpu().numpy()
        bsp.accumulate_weights(q.cuda(), lse, k, w, t.kv_indptr, t.kv_indices, t.last_page_len, qo_indptr=t.qo_indptr, decay=0.75,
                               k_exp=exps.get("k_exp"))
        host = b.kv_indptr, b.kv_indices, b.last_page_len
        l64 = lse.cpu().numpy()
        want, size = ev.weights(q.double().numpy(), l64.astype(np.float64), kv64[0], was, b.qo_indptr, *host, scale, decay=0.75)
        got = w.cpu().numpy()
        used = size > 0
        assert not np.isnan(got[used]).any() and np.array_equal(np.isnan(got), np.isnan(want))
        assert (np.abs(got - want)[used] <= bound(b, kv64[0], l64, scale, size, 0.0)[used]).all()
        # the choice and the move
        kept, n_new = bsp.select_tokens(w, t.kv_indptr, t.kv_indices, t.last_page_len, dev(np.array(budget, np.int32)), 100, 2, 4)
        K, N = ev.select(got, *host, budget, 100, 2, 4)
        assert np.array_equal(kept.cpu().numpy(), K) and np.array_equal(n_new.cpu().numpy(), N)
        rows = [(raw(c), e.cpu().numpy()) for c, e in zip((k, v), exps.values())] if f8 else [raw(c) for c in (k, v)]
        bsp.compact_cache(kept, n_new, t.kv_indptr, t.kv_indices, t.last_page_len, k, v, weights=w, **exps)
        torch.cuda.synchronize()
        for i, c in enumerate((k, v)):
            if f8:
                moved, me = ev.compact_codes(*rows[i], K, N, b.kv_indptr, b.kv_indices, PS, kc.encode)
                assert np.array_equal(list(exps.values())[i].cpu().numpy(), me)
            else:
                moved = ev.compact(rows[i], K, N, b.kv_indptr, b.kv_indices, PS)
            assert np.array_equal(raw(c), moved)
        moved = ev.compact(np.swapaxes(got, 1, 2), K, N, b.kv_indptr, b.kv_indices, PS).swapaxes(1, 2)
        assert np.array_equal(w.cpu().numpy(), moved, equal_nan=True)
        # the pages behind the kept tokens are free again
        keep_pages = -(-N // PS)
        freed = [b.kv_indices[b.kv_indptr[i] + keep_pages[i]:b.kv_indptr[i + 1]] for i in range(B)]
        pool, lens = np.concatenate(freed + [pool]).astype(np.int32), N.astype(np.int64)
