"""What bsp_check_weights_wait refuses on the host (argument checks run before any device call; the pointers are never
followed)."""
import ctypes

import pytest

P16 = ctypes.c_void_p(4096)


@pytest.fixture(scope="module")
def native():
    from block_sparse_paged_gb300 import build
    build.build()
    from block_sparse_paged_gb300 import _native
    _native.load()
    return _native


def check(native, **kw):
    pr = dict(mode=0, num_qo_heads=8, num_kv_heads=2, head_dim=128, page_size=16, causal=0, dtype=0, window_left=-1, logits_soft_cap=0.0)
    a = dict(q=P16, lse=P16, n=4, k=P16, ke=None, pages=9, w=P16, batch=4, qo=P16, kvp=P16, kvi=P16, cap=9, last=P16, scale=0.1,
             decay=1.0, limit=1000)
    for key, v in kw.items():
        (pr if key in pr else a)[key] = v
    return native.load().bsp_check_weights_wait(ctypes.byref(native.Problem(*pr.values())), *a.values(), None)


@pytest.mark.parametrize("kw", [dict(limit=0), dict(limit=-5), dict(limit=(1 << 33) + 1), dict(q=None), dict(w=None), dict(decay=-1.0),
                                dict(batch=-1), dict(num_qo_heads=7)], ids=str)
def test_refuses(native, kw):
    assert check(native, **kw) == native.BSP_ERR_INVALID_ARG
    assert native.load().bsp_last_error()


@pytest.mark.parametrize("kw", [dict(dtype=1), dict(head_dim=64), dict(window_left=5), dict(logits_soft_cap=3.0)], ids=str)
def test_unsupported(native, kw):
    assert check(native, **kw) == native.BSP_ERR_UNSUPPORTED


def test_nothing(native):
    assert check(native, batch=0) == native.BSP_OK and check(native, cap=0) == native.BSP_OK
