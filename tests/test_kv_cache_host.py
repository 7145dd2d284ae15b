"""The 8-bit KV cache on the host: the oracle's append and tables against facts
worked out by hand, and what the entry points refuse (argument checks run before
any device call; the pointers here are never followed)."""
import ctypes

import numpy as np
import pytest

import oracle
from oracle import kv_cache as kc


@pytest.fixture(scope="module")
def native():
    from block_sparse_paged_gb300 import build
    build.build()
    from block_sparse_paged_gb300 import _native
    _native.load()
    return _native


# ---- oracle pins ---------------------------------------------------------------
def test_encode_is_the_nearest_code_with_ties_to_even():
    vals = np.array([oracle.fp8.e4m3_value(c) for c in range(127)])
    assert np.array_equal(kc.encode(vals), np.arange(127))           # every code maps to itself
    assert np.array_equal(kc.encode(-vals[1:]), np.arange(1, 127) + 128)
    mid = (vals[1:] + vals[:-1]) / 2
    even = np.where(np.arange(126) % 2 == 0, np.arange(126), np.arange(1, 127))
    assert np.array_equal(kc.encode(mid), even)                      # ties
    assert np.array_equal(kc.encode(np.nextafter(mid, 0)), np.arange(126))
    assert np.array_equal(kc.encode(np.nextafter(mid, 1e9)), np.arange(1, 127))
    assert list(kc.encode(np.array([1e30, np.inf, np.nan, -500.0]))) == [126, 127, 127, 254]


@pytest.mark.parametrize("amax,e", [(448.0, 0), (448.0001, 1), (224.0, -1), (1.0, -8), (0.875, -9), (0.0, -117),
                                    (2.0 ** -140, -117), (3.3e38, 119), (1.75, -8), (1.7500001, -7)])
def test_exponent(amax, e):
    assert kc.exponent_for(amax) == e


def test_append_rescales_what_a_page_held():
    codes = np.zeros((2, 4, 1, 2), np.uint8)
    exps = np.full((2, 1), -5, np.int8)
    codes[1, :2, 0] = kc.encode(np.array([[448.0, 1.0], [-2.0, 2.0 ** -9]]))
    x = np.array([[[56.0, 0.0]]])                                   # needs exponent -3
    c, e = kc.append(x, [6], codes, exps)
    assert list(e[:, 0]) == [-5, -3]
    got = kc.values(c, e)[1, :, 0]
    assert got[0].tolist() == [14.0, 1.0 / 32] and got[1].tolist() == [-1 / 16, 0.0]  # 2^-14 -> tie to zero
    assert got[2].tolist() == [56.0, 0.0] and np.array_equal(c[0], codes[0])


def test_tables_worked_example():
    bt = np.array([[7, 3, -1], [-1, -1, -1], [2, -1, -1]], np.int32)
    t = kc.tables([5, 0, 3], [4, 0, 1], [9, 8, 1], 3, bt, 4, 6, 7)
    assert t["block_table"].tolist() == [[7, 3, 9], [-1, -1, -1], [2, -1, -1]]
    assert t["kv_indptr"].tolist() == [0, 3, 3, 4] and t["last_page_len"].tolist() == [1, 0, 4]
    assert t["kv_indices"].tolist() == [7, 3, 9, 2, 0, 0] and t["qo_indptr"].tolist() == [0, 4, 4, 5]
    assert t["slot_map"].tolist() == [13, 14, 15, 36, 11, -1, -1]
    assert t["positions"].tolist() == [5, 6, 7, 8, 3, 0, 0] and t["counts"].tolist() == [4, 5, 1, 0]


# ---- refusals ------------------------------------------------------------------
A = 256  # an aligned address that is never followed


def tables_args(**kw):
    d = dict(batch=2, ps=16, cached=A, new=A, free=A, free_cap=8, num_free=A, table=A, stride=4, width=4, kvp=A, last=A,
             idx=A, cap_pages=8, qop=A, slots=A, pos=A, cap_tok=8, counts=A)
    d.update(kw)
    return list(d.values()) + [None]


@pytest.mark.parametrize("kw", [dict(batch=-1), dict(ps=0), dict(free_cap=-1), dict(cap_pages=-1), dict(cap_tok=-1),
                                dict(width=-1), dict(stride=3), dict(cached=None), dict(new=None), dict(table=None),
                                dict(num_free=None), dict(free=None), dict(idx=None), dict(slots=None), dict(pos=None),
                                dict(counts=None), dict(kvp=None), dict(qop=None), dict(last=None),
                                dict(cap_tok=1 << 31), dict(slots=A + 8), dict(idx=A + 4), dict(pos=A + 4)],
                         ids=lambda kw: "_".join(kw))
def test_tables_refuse(native, kw):
    lib = native.load()
    assert lib.bsp_build_page_tables(*tables_args(**kw)) == native.BSP_ERR_INVALID_ARG
    assert lib.bsp_last_error()


def test_tables_refuse_a_batch_past_shared_memory(native):
    assert native.load().bsp_build_page_tables(*tables_args(batch=16385)) == native.BSP_ERR_UNSUPPORTED


def append_args(**kw):
    d = dict(k=A, v=A, kt=1024, kh=128, vt=1024, vh=128, dtype=0, n=3, slots=A, kp=A, vp=A, ke=A, ve=A, pages=4, ps=16,
             H=8, D=128)
    d.update(kw)
    return list(d.values()) + [None]


@pytest.mark.parametrize("kw", [dict(k=None), dict(v=None), dict(slots=None), dict(kp=None), dict(vp=None),
                                dict(ke=None), dict(ve=None), dict(n=-1), dict(pages=0), dict(ps=0), dict(H=0),
                                dict(dtype=7), dict(k=A + 2), dict(v=A + 8), dict(kp=A + 4), dict(kt=1025),
                                dict(vh=132, dtype=0), dict(pages=1 << 31)], ids=lambda kw: "_".join(kw))
def test_append_refuses(native, kw):
    assert native.load().bsp_append_kv_fp8(*append_args(**kw)) == native.BSP_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(D=64), dict(D=256), dict(H=40000), dict(pages=1 << 28), dict(n=1 << 31)])
def test_append_unsupported(native, kw):
    assert native.load().bsp_append_kv_fp8(*append_args(**kw)) == native.BSP_ERR_UNSUPPORTED


def test_append_of_nothing_is_fine(native):
    assert native.load().bsp_append_kv_fp8(*append_args(n=0, k=None, slots=None)) == native.BSP_OK


def test_python_entries_refuse_host_tensors(native):
    import torch
    import block_sparse_paged_gb300 as bsp
    i32 = torch.int32
    z = torch.zeros(2, dtype=i32)
    with pytest.raises(ValueError, match="block_table"):
        bsp.build_page_tables(z, z, z, z[:1], torch.zeros(2, 3, dtype=i32), 16, 4, 4)
    p = torch.zeros(2, 4, 1, 128).to(torch.float8_e4m3fn)
    e = torch.zeros(2, 1, dtype=torch.int8)
    k = torch.zeros(1, 1, 128, dtype=torch.bfloat16)
    for bad in (lambda: bsp.append_kv(k, k, torch.zeros(1, dtype=torch.int64), p, p, e, e),
                lambda: bsp.append_kv(k[:, :, ::2], k[:, :, ::2], torch.zeros(1, dtype=torch.int64), p, p, e, e),
                lambda: bsp.append_kv(k, k.float(), torch.zeros(1, dtype=torch.int64), p, p, e, e),
                lambda: bsp.append_kv(k, k, torch.zeros(2, dtype=torch.int64), p, p, e, e),
                lambda: bsp.append_kv(k, k, torch.zeros(1, dtype=torch.int64), p, p, e[:1], e)):
        with pytest.raises(ValueError):
            bad()


# ---- attention over the cache ----------------------------------------------------
def block_plan(mode, H=8, Hkv=2, D=128, dtype=None):
    """A plan info that claims to be copied to a device (the checks need no more)."""
    import torch
    import block_sparse_paged_gb300 as bsp
    prob = bsp.make_problem(mode, H, Hkv, D, 16, False, dtype or torch.bfloat16)
    cap = bsp.Capacity(2, 4, 64, 1, 0, 0)
    info = bsp.plan_host(prob, cap, [0, 2, 3], [3, 16], [0, 1, 2])[0]
    info.valid = 1
    return info


def run_args(info, **kw):
    d = dict(q=A, k=A, v=A, ke=A, ve=A, idx=A, pages=4, scale=0.1, o=A, lse=None, ws=A)
    d.update(kw)
    a = [ctypes.byref(info)] + list(d.values()) + [None]
    a[-2:-2] = [None, 0]  # no region
    return a


@pytest.mark.parametrize("mode", [0, 1])
@pytest.mark.parametrize("kw", [dict(q=None), dict(k=None), dict(v=None), dict(ke=None), dict(ve=None), dict(idx=None),
                                dict(pages=0), dict(pages=-1), dict(pages=1 << 31), dict(o=None), dict(ws=None),
                                dict(q=A + 8), dict(k=A + 4), dict(o=A + 2)], ids=lambda kw: "_".join(kw))
def test_block_runs_refuse(native, mode, kw):
    lib = native.load()
    fn = lib.bsp_decode_run_fp8_block if mode == 0 else lib.bsp_prefill_run_fp8_block
    assert fn(*run_args(block_plan(mode), **kw)) == native.BSP_ERR_INVALID_ARG


@pytest.mark.parametrize("scale,modes", [(float("nan"), (0, 1)), (float("inf"), (0, 1)), (0.0, (1,)), (-1.0, (1,))])
def test_block_runs_refuse_scales(native, scale, modes):
    lib = native.load()
    for mode in modes:
        fn = lib.bsp_decode_run_fp8_block if mode == 0 else lib.bsp_prefill_run_fp8_block
        assert fn(*run_args(block_plan(mode), scale=scale)) == native.BSP_ERR_INVALID_ARG


@pytest.mark.parametrize("mode", [0, 1])
def test_block_runs_refuse_plans(native, mode):
    import torch
    lib = native.load()
    fn = lib.bsp_decode_run_fp8_block if mode == 0 else lib.bsp_prefill_run_fp8_block
    other = block_plan(mode)
    other.problem.mode = 1 - mode
    args = run_args(block_plan(mode))
    assert fn(ctypes.byref(other), *args[1:]) == native.BSP_ERR_INVALID_ARG       # the other mode's plan
    host = block_plan(mode)
    host.valid = 2
    assert fn(*run_args(host)) == native.BSP_ERR_INVALID_ARG                      # a host-only plan
    if mode == 0:
        assert fn(*run_args(block_plan(0, D=64))) == native.BSP_ERR_UNSUPPORTED
        assert fn(*run_args(block_plan(0, dtype=torch.float32))) == native.BSP_ERR_UNSUPPORTED


def test_region_size_and_refusals(native):
    """A region is wanted where query tiles read cached tokens often enough, and must hold the page table."""
    lib = native.load()
    info = block_plan(1, H=8, Hkv=2)
    assert lib.bsp_prefill_fp8_region_size(ctypes.byref(info)) == 0               # one tile per request
    import torch
    import block_sparse_paged_gb300 as bsp
    prob = bsp.make_problem(1, 8, 2, 128, 16, True, torch.bfloat16)
    big = bsp.plan_host(prob, bsp.Capacity(2, 4, 900, 1, 0, 0), [0, 32], [16], [0, 512])[0]
    assert lib.bsp_prefill_fp8_region_size(ctypes.byref(big)) == 512 * 2 * 512    # tokens x heads x 4 bytes x 128
    big.valid = 1
    for region, nbytes, rc in ((A, 512 * 2 * 512 - 1, native.BSP_ERR_CAPACITY), (A + 16, 1 << 30, native.BSP_ERR_INVALID_ARG)):
        a = run_args(big)
        a[-4:-2] = [region, nbytes]
        assert lib.bsp_prefill_run_fp8_block(*a) == rc
    assert lib.bsp_prefill_fp8_region_size(ctypes.byref(block_plan(0))) == 0


def test_decode_region_size_and_refusals(native):
    """A region is wanted for pages of one or two tokens and work enough, and must hold the page table."""
    import torch
    import block_sparse_paged_gb300 as bsp
    lib = native.load()
    assert lib.bsp_decode_fp8_region_size(ctypes.byref(block_plan(0))) == 0
    assert lib.bsp_decode_fp8_region_size(ctypes.byref(block_plan(1))) == 0

    def plan(ps, tokens):
        prob = bsp.make_problem(0, 8, 2, 128, ps, False, torch.bfloat16)
        info = bsp.plan_host(prob, bsp.Capacity(1, 2, 1, 1, 0, 0), [0, -(-tokens // ps)], [(tokens - 1) % ps + 1], [0, 1])[0]
        info.valid = 1
        return info
    assert lib.bsp_decode_fp8_region_size(ctypes.byref(plan(3, 9000))) == 0
    assert lib.bsp_decode_fp8_region_size(ctypes.byref(plan(2, 5000))) == 0
    assert lib.bsp_decode_fp8_region_size(ctypes.byref(plan(2, 9000))) == 4512 * 2 * 2
    assert lib.bsp_decode_fp8_region_size(ctypes.byref(plan(1, 2000))) == 0      # 2000 x 2 heads on 2 CTAs
    big = plan(1, 2570)
    assert lib.bsp_decode_fp8_region_size(ctypes.byref(big)) == 2576 * 2 * 2     # whole 16s x K, V x heads
    for region, nbytes, rc in ((A, 2576 * 4 - 1, native.BSP_ERR_CAPACITY), (A + 8, 1 << 30, native.BSP_ERR_INVALID_ARG)):
        a = run_args(big)
        a[-4:-2] = [region, nbytes]
        assert lib.bsp_decode_run_fp8_block(*a) == rc


def test_region_of_pages_past_the_conversion_kernel(native):
    """Pages of 2^28 rows over all heads (32-bit vector counts): converted inside only."""
    import torch
    import block_sparse_paged_gb300 as bsp
    lib = native.load()
    prob = bsp.make_problem(1, 64, 2, 128, 1 << 27, True, torch.bfloat16)
    info = bsp.plan_host(prob, bsp.Capacity(1, 2, 1 << 20, 1, 0, 0), [0, 1], [1 << 27], [0, 1 << 20])[0]
    info.valid = 1
    assert lib.bsp_prefill_fp8_region_size(ctypes.byref(info)) == 0
    a = run_args(info)
    a[-4:-2] = [A, 1 << 38]
    assert lib.bsp_prefill_run_fp8_block(*a) == native.BSP_ERR_UNSUPPORTED
