"""What the rounding of P takes in differential attention: with lambda 1 and two maps that nearly agree, the output is a small
difference of two averages, and P's rounding stands out of it where it is not kept. The bound (derived beside `check`) has no
room for a P of eight bits."""
import numpy as np
import pytest
import torch

from gpu_helpers import lib
from oracle import evict as ev
from test_gpu_differential import Run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bsp():
    return lib()


def near_equal_maps(bsp, qo, kv, mode, ps, **kw):
    """Small scores (weights of a row within a few percent), the second halves of the keys a quarter of a step off the first."""
    r = Run(bsp, 61, qo, kv, 8, 2, ps, mode=mode, lam=1.0, **kw)
    q = r.b.q.float() * 0.02
    q[..., 64:] = q[..., :64]
    k = r.b.k_pages.float()
    k[..., 64:] = k[..., :64] + 0.25 * k[..., 64:]
    r.b.q, r.b.k_pages = q.bfloat16(), k.bfloat16()
    r.q, r.k, r.k64 = r.b.q.cuda(), r.b.k_pages.cuda(), r.b.k_pages.double().numpy()
    return r


def check(r, out):
    """A score is off by e = 68 s 2^-23 + 2^-20, s >= sum |q k| / 8 over a half (64 products in fp32, scaled, moved by the maximum
    and exponentiated), a weight by e and by its sum's e relatively; P is kept to 2^-16 of itself (its eight bits and eight of what
    they leave), and the sums over n keys take 2^-23 each. The maps add up in `size`; the output is rounded once, 2^-8."""
    torch.cuda.synchronize()
    assert r.pa.check_device_error() == 0
    b, q = r.b, r.b.q.double().numpy()
    o, _, size = ev.differential(q, np.nan_to_num(r.k64), np.nan_to_num(r.v64), b.qo_indptr, b.kv_indptr, b.kv_indices, b.last_page_len, 0.125, np.ones(8))
    s = 0.125 * np.abs(q[..., :64]).sum(axis=2).max() * np.nanmax(np.abs(r.k64))
    n = int(ev.lengths(b.kv_indptr, b.last_page_len, b.page_size).max())
    d = size * (2 * (s * 68 * 2.0 ** -23 + 2.0 ** -20) + 2.0 ** -16 + n * 2.0 ** -23)
    off = np.abs(out.double().cpu().numpy() - o)
    assert (off <= d + 2.0 ** -8 * (np.abs(o) + d)).all(), ((off - d).max(), (off / size).max())


@pytest.mark.parametrize("ps", [1, 16])
@pytest.mark.parametrize("num_ctas", [None, 3])
def test_decode(bsp, ps, num_ctas):
    r = near_equal_maps(bsp, [1] * 4, [64, 200, 130, 300], "decode", ps, num_ctas=num_ctas)
    check(r, r(return_lse=False))


@pytest.mark.parametrize("ps", [1, 16, 128])
@pytest.mark.parametrize("qo,kv", [([64], [64]), ([40, 100], [120, 128]), ([150, 20], [300, 260])], ids=str)
def test_prefill(bsp, ps, qo, kv):
    """Keys in the first half of a tile, in both, and over several tiles."""
    r = near_equal_maps(bsp, qo, kv, "prefill", ps, num_ctas=1)  # (an item holds all keys that its queries see)
    assert r.pa.info.num_merges == 0
    check(r, r(return_lse=False))


def test_prefill_split_outputs(bsp):
    r = near_equal_maps(bsp, [64, 5], [300, 290], "prefill", 16, num_ctas=16, chunks_per_cta=2)
    assert r.pa.info.num_merges > 0
    check(r, r(return_lse=False))
