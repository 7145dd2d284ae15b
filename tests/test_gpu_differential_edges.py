"""Differential attention at the edges: queries of NaN."""
import pytest
import torch

from gpu_helpers import lib
from test_gpu_differential import Run

pytestmark = pytest.mark.gpu
MODES = pytest.mark.parametrize("mode", ["decode", "prefill"])
POOLS = pytest.mark.parametrize("f8", [False, True], ids=["bf16", "e4m3"])


@pytest.fixture(scope="module")
def bsp():
    return lib()


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
