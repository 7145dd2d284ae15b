"""Differential attention on the host: what its entry points refuse (argument checks run before any device call; the
device pointers here are never followed) and what its plan is."""
import ctypes

import numpy as np
import pytest

P16 = ctypes.c_void_p(4096)


@pytest.fixture(scope="module")
def native():
    from block_sparse_paged_gb300 import build
    build.build()
    from block_sparse_paged_gb300 import _native
    _native.load()
    return _native


def planned(native, mode, heads=32, kv=8, D=128, ps=16, dtype=0, pages=4):
    """A host plan over `heads` maps, marked as copied (the checks come before anything reads the copy)."""
    lib = native.load()
    prob, cap = native.Problem(mode, heads, kv, D, ps, mode, dtype), native.Capacity(2, 16, 64)
    staging = np.zeros(lib.bsp_host_staging_size(ctypes.byref(prob), ctypes.byref(cap)), np.uint8)
    i32 = lambda *a: np.array(a, np.int32).ctypes.data_as(ctypes.c_void_p)  # noqa: E731
    keep = [np.array([0, 1, 2], np.int32), np.array([0, pages // 2, pages], np.int32), np.array([3, 5] if pages else [0, 0], np.int32)]
    info = native.PlanInfo()
    native.check(lib.bsp_plan(ctypes.byref(prob), ctypes.byref(cap), 2, *(x.ctypes.data_as(ctypes.c_void_p) for x in keep), 2, 1,
                              staging.ctypes.data_as(ctypes.c_void_p), None, 0, None, ctypes.byref(info)))
    info.valid = 1
    del i32
    return info


def run(native, mode, info=None, lam=4096, norm=None, eps=1e-5, out=1.0, **kw):
    a = dict(q=P16, k=P16, v=P16, ke=None, ve=None, idx=P16, pages=9, scale=0.1, o=P16, lse=P16, region=None, nbytes=0, ws=P16)
    a.update(kw)
    d = native.Differential(lam, norm, eps, out)
    info = info or planned(native, mode)
    fn = native.load().bsp_prefill_run_diff if mode else native.load().bsp_decode_run_diff
    return fn(ctypes.byref(info), ctypes.byref(d), *a.values(), None)


@pytest.mark.parametrize("mode", [0, 1], ids=["decode", "prefill"])
@pytest.mark.parametrize("kw", [
    dict(lam=None), dict(norm=4100), dict(eps=-1.0), dict(eps=float("nan")), dict(out=float("inf")), dict(q=None), dict(k=None),
    dict(v=None), dict(o=None), dict(ws=None), dict(idx=None), dict(pages=0), dict(scale=float("nan")), dict(ke=P16), dict(ve=P16),
    dict(q=ctypes.c_void_p(4104)), dict(lse=ctypes.c_void_p(4100)), dict(ke=P16, ve=P16, region=ctypes.c_void_p(4104), nbytes=1 << 20)], ids=str)
def test_refuses(native, mode, kw):
    assert run(native, mode, **kw) == native.BSP_ERR_INVALID_ARG
    assert native.load().bsp_last_error()


@pytest.mark.parametrize("mode", [0, 1], ids=["decode", "prefill"])
def test_refuses_plans(native, mode):
    assert run(native, mode, planned(native, 1 - mode)) == native.BSP_ERR_INVALID_ARG     # the other mode's
    assert run(native, mode, planned(native, mode, heads=8)) == native.BSP_ERR_INVALID_ARG  # one map per kv head
    info = planned(native, mode)
    info.problem.sink = 4096
    assert run(native, mode, info) == native.BSP_ERR_UNSUPPORTED
    info = planned(native, mode)
    info.valid = 2
    assert run(native, mode, info) == native.BSP_ERR_INVALID_ARG
    assert run(native, mode, planned(native, mode, D=64)) == native.BSP_ERR_UNSUPPORTED
    assert run(native, 0, planned(native, 0, dtype=1)) == native.BSP_ERR_UNSUPPORTED


def test_regions(native):
    lib = native.load()
    pre = planned(native, 1)
    assert lib.bsp_prefill_diff_region_size(ctypes.byref(pre)) == 4 * 16 * 8 * 512
    assert lib.bsp_prefill_diff_region_size(ctypes.byref(planned(native, 0))) == 0
    assert lib.bsp_prefill_diff_region_size(ctypes.byref(planned(native, 1, pages=0))) == 0
    assert run(native, 1, ke=P16, ve=P16) == native.BSP_ERR_INVALID_ARG  # no region
    assert run(native, 1, ke=P16, ve=P16, region=P16, nbytes=100) == native.BSP_ERR_CAPACITY
    assert run(native, 0, ke=P16, ve=P16, region=P16, nbytes=8) == native.BSP_ERR_CAPACITY


def test_struct_matches_header(native, tmp_path):
    import os
    import subprocess

    from conftest import ROOT
    src = tmp_path / "d.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "bsp.h"\nint main(void) { printf("%zu %zu %zu\\n", '
                   'sizeof(bsp_differential), offsetof(bsp_differential, norm_eps), offsetof(bsp_differential, out_scale)); return 0; }')
    subprocess.check_call(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(tmp_path / "d")])
    D = native.Differential
    assert [int(x) for x in subprocess.check_output([str(tmp_path / "d")]).split()] == [ctypes.sizeof(D), D.norm_eps.offset, D.out_scale.offset]
