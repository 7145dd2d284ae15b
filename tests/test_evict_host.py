"""Eviction by gathered weight on the host: the oracle against facts worked out by hand, and what the entry points refuse
(argument checks run before any device call; the pointers here are never followed)."""
import ctypes

import numpy as np
import pytest

from oracle import evict as ev
from oracle import kv_cache as kc


@pytest.fixture(scope="module")
def native():
    from block_sparse_paged_gb300 import build
    build.build()
    from block_sparse_paged_gb300 import _native
    _native.load()
    return _native


# ---- oracle pins ---------------------------------------------------------------
def test_weights_worked_example():
    # one head, D = 2, page size 2: three keys, the last is the query's own; scores 0, log 2, log 5 -> weights 1/8, 2/8, 5/8
    k = np.zeros((2, 2, 1, 2))
    k[1, 0, 0], k[1, 1, 0], k[0, 0, 0] = [0, 0], [np.log(2), 0], [np.log(5), 0]
    q = np.array([[[1.0, 7.0]]])
    w = np.full((2, 1, 2), 10.0)
    got, _ = ev.weights(q, np.array([[np.log(8)]]), k, w, [0, 1], [0, 2], [1, 0], [1], 1.0, decay=0.5)
    assert np.allclose(got[1, 0], [5 + 1 / 8, 5 + 2 / 8]) and np.allclose(got[0, 0], [5 / 8, 10.0])


def test_differential_worked_example():
    # D = 2: halves of one value; map 1 weighs the two keys 1/2 and 1/2, map 2 1/3 and 2/3
    k = np.array([[[[0.0, 0.0]]], [[[0.0, np.log(2)]]]])
    v = np.array([[[[6.0, 0.0]]], [[[0.0, 6.0]]]])
    o, lse, _ = ev.differential(np.array([[[3.0, 1.0]]]), k, v, [0, 1], [0, 2], [0, 1], [1], 1.0, [0.5])
    assert np.allclose(o[0, 0], [3 - 0.5 * 2, 3 - 0.5 * 4]) and np.allclose(lse[0, 0], [np.log(2), np.log(3)])
    n, _, _ = ev.differential(np.array([[[3.0, 1.0]]]), k, v, [0, 1], [0, 2], [0, 1], [1], 1.0, [0.5], norm=np.array([1.0, 2.0]),
                              eps=0.0, out_scale=3.0)
    assert np.allclose(n[0, 0], 3 * np.array([2.0, 1.0 * 2]) / np.sqrt(2.5))


def test_select_worked_example():
    w = np.array([5.0, 1, 9, 1, np.nan, 1, 0, 0]).reshape(4, 1, 2)
    kept, n = ev.select(w, [0, 4], [0, 1, 2, 3], [2], [5], 6, 1, 1)
    assert n.tolist() == [5] and kept[0, 0].tolist() == [0, 1, 2, 3, 7, -1]


def test_compact_worked_example():
    rows = np.arange(6).reshape(3, 2, 1)
    out = ev.compact(rows, np.array([[[0, 2, 5]]]), [3], [0, 3], [2, 0, 1], 2)
    assert out[2, :, 0].tolist() == [4, 0] and out[0, :, 0].tolist() == [3, 1] and out[1, :, 0].tolist() == [2, 3]
    codes = kc.encode(np.array([8.0, 3.0, 1.0, 2.0])).reshape(2, 2, 1, 1)
    c, e = ev.compact_codes(codes, np.array([[-1], [3]], np.int8), np.array([[[1, 2]]]), [2], [0, 2], [0, 1], 2, kc.encode)
    assert e[:, 0].tolist() == [3, 3] and kc.values(c, e)[0, :, 0, 0].tolist() == [1.5, 8.0]


# ---- refusals ------------------------------------------------------------------
P16 = ctypes.c_void_p(4096)


def accumulate(native, **kw):
    pr = dict(mode=0, num_qo_heads=8, num_kv_heads=2, head_dim=128, page_size=16, causal=0, dtype=0, window_left=-1,
              logits_soft_cap=0.0)
    a = dict(q=P16, lse=P16, n=4, k=P16, ke=None, pages=9, w=P16, batch=4, qo=P16, kvp=P16, kvi=P16, cap=9, last=P16,
             scale=0.1, decay=1.0, lam=None)
    for key, v in kw.items():
        (pr if key in pr else a)[key] = v
    prob = native.Problem(*pr.values())
    return native.load().bsp_accumulate_weights(ctypes.byref(prob), *a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(num_qo_heads=7), dict(page_size=0), dict(dtype=3), dict(batch=-1), dict(batch=70000), dict(pages=0), dict(cap=-1),
    dict(scale=float("nan")), dict(decay=-0.5), dict(decay=float("inf")), dict(n=-1), dict(q=None), dict(lse=None),
    dict(k=None), dict(w=None), dict(kvp=None), dict(kvi=None), dict(last=None), dict(k=ctypes.c_void_p(4104)),
    dict(q=ctypes.c_void_p(4098)), dict(logits_soft_cap=-1.0), dict(n=1 << 31), dict(lam=P16, lse=ctypes.c_void_p(4100))], ids=str)
def test_accumulate_refuses(native, kw):
    assert accumulate(native, **kw) == native.BSP_ERR_INVALID_ARG
    assert native.load().bsp_last_error()


@pytest.mark.parametrize("kw", [
    dict(head_dim=96), dict(dtype=1, head_dim=48), dict(dtype=1, lam=P16), dict(dtype=1, ke=P16), dict(head_dim=64, ke=P16),
    dict(num_qo_heads=40000, num_kv_heads=40000), dict(pages=1 << 28), dict(cap=1 << 30, page_size=4096, pages=16)], ids=str)
def test_accumulate_unsupported(native, kw):
    assert accumulate(native, **kw) == native.BSP_ERR_UNSUPPORTED


def test_nothing_to_accumulate(native):
    assert accumulate(native, batch=0, kvp=None, kvi=None, last=None, q=None, lse=None, n=0) == native.BSP_OK
    assert accumulate(native, cap=0, kvi=None) == native.BSP_OK


def test_accumulate_does_not_read_the_other_members(native):
    """The mode, causal and sink of the problem say nothing here."""
    for kw in (dict(mode=5), dict(causal=7), dict(causal=-1), dict(mode=1, num_qo_heads=12)):
        assert accumulate(native, batch=0, **kw) == native.BSP_OK


def select(native, **kw):
    a = dict(w=P16, pages=9, ps=16, H=2, batch=4, kvp=P16, kvi=P16, cap=9, last=P16, budget=P16, most=8, sinks=1, recent=2,
             kept=P16, new=P16)
    a.update(kw)
    return native.load().bsp_select_tokens(*a.values(), None)


@pytest.mark.parametrize("kw", [dict(w=None), dict(pages=0), dict(ps=0), dict(H=0), dict(batch=-1), dict(kvp=None),
                                dict(kvi=None), dict(last=None), dict(budget=None), dict(most=-1), dict(sinks=-1),
                                dict(recent=-1), dict(kept=None), dict(new=None), dict(cap=-3)], ids=str)
def test_select_refuses(native, kw):
    assert select(native, **kw) == native.BSP_ERR_INVALID_ARG


def test_select_nothing(native):
    assert select(native, batch=0, kvp=None, kvi=None, last=None, budget=None, new=None) == native.BSP_OK
    assert select(native, batch=60000, H=30000) == native.BSP_ERR_UNSUPPORTED


def compact(native, **kw):
    a = dict(kept=P16, new=P16, most=8, batch=4, kvp=P16, kvi=P16, cap=9, last=P16, k=P16, v=P16, ke=None, ve=None, w=None,
             pages=9, ps=16, H=2, row=256)
    a.update(kw)
    return native.load().bsp_compact_cache(*a.values(), None)


@pytest.mark.parametrize("kw", [dict(kept=None), dict(new=None), dict(most=-1), dict(batch=-1), dict(kvp=None), dict(k=None),
                                dict(v=None), dict(ke=P16), dict(ve=P16), dict(row=0), dict(row=24), dict(pages=0),
                                dict(k=ctypes.c_void_p(4104))], ids=str)
def test_compact_refuses(native, kw):
    assert compact(native, **kw) == native.BSP_ERR_INVALID_ARG


def test_compact_unsupported_and_nothing(native):
    assert compact(native, ke=P16, ve=P16) == native.BSP_ERR_UNSUPPORTED  # 256-byte rows of e4m3
    assert compact(native, ke=P16, ve=P16, row=128, ps=4097) == native.BSP_ERR_UNSUPPORTED
    assert compact(native, batch=0, kept=None, new=None, kvp=None, kvi=None, last=None) == native.BSP_OK
    assert compact(native, most=0, kept=None) == native.BSP_OK
