"""Outputs that a call allocates for itself belong to the stream that it runs on: memory that the current stream still
uses is not taken for them."""
import pytest
import torch

import workloads
from gpu_helpers import lib, to_dev
from test_gpu_fp8_block import cache8

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def bsp():
    return lib()


def freed_while_in_use(shape, dtype, call):
    """call(stream) while a copy of a tensor of the call's output size, freed on the host already, still waits on the
    current stream; returns the call's result and whether the copy got the tensor's values."""
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    x = torch.full(shape, 3, dtype=dtype, device="cuda")
    y = torch.zeros_like(x)
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)  # about 0.1 s
    y.copy_(x)
    del x
    out = call(s)
    torch.cuda.synchronize()
    return out, bool((y == 3).all())


def attention(bsp, mode, fp8):
    qo = [1] * 600 if mode == "decode" else [300, 300]
    kv = [33] * 600 if mode == "decode" else [300, 300]
    b = workloads.paged_batch(321, qo, kv, 32, 8, 128, 16, "bf16", causal=mode == "prefill")
    pa = bsp.PagedAttention(mode, 32, 8, 128, 16, mode == "prefill", torch.bfloat16, max_batch=b.batch, max_qo_tokens=600)
    pa.plan(b.kv_indptr, b.last_page_len, qo_indptr=b.qo_indptr)
    q, k, v, idx = to_dev(b)
    kw = {}
    if fp8:
        k8, ke, v8, ve = (torch.from_numpy(a).cuda() for a in cache8(b, 321))
        k, v, kw = k8.view(F8), v8.view(F8), dict(k_exp=ke, v_exp=ve)
    return q, lambda stream=None: pa.run(q, k, v, idx, stream=stream, **kw)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("mode", ["decode", "prefill"])
@pytest.mark.parametrize("which", ["out", "lse"])
def test_attention(bsp, mode, fp8, which):
    q, run = attention(bsp, mode, fp8)
    want = [t.clone() for t in run()]
    shape, dtype = (q.shape, torch.bfloat16) if which == "out" else (q.shape[:2], torch.float32)
    got, kept = freed_while_in_use(shape, dtype, run)
    assert kept
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_page_tables(bsp):
    B, ps, n = 4, 16, 40000
    i32 = dict(dtype=torch.int32, device="cuda")
    cached, new = torch.zeros(B, **i32), torch.full((B,), n // B, **i32)
    free, nfree = torch.arange(4000, **i32), torch.tensor([4000], **i32)
    table = torch.full((B, 1000), -1, **i32)

    def call(stream=None):
        return bsp.build_page_tables(cached, new, free, nfree, table, ps, 4000, n, stream=stream)
    want = call()
    torch.cuda.synchronize()
    for shape, dtype in (((n,), torch.int64), ((want._ints.numel(),), torch.int32)):
        got, kept = freed_while_in_use(shape, dtype, call)
        assert kept
        assert all(torch.equal(getattr(got, f), getattr(want, f)) for f in want._fields)


def test_merge_state(bsp):
    rng = torch.Generator().manual_seed(5)
    o = [torch.randn(600, 32, 128, generator=rng).bfloat16().cuda() for _ in range(2)]
    l = [torch.randn(600, 32, generator=rng).cuda() for _ in range(2)]
    call = lambda stream=None: bsp.merge_state(o[0], l[0], o[1], l[1], stream=stream)  # noqa: E731
    want = [t.clone() for t in call()]
    for shape, dtype in ((o[0].shape, torch.bfloat16), (l[0].shape, torch.float32)):
        got, kept = freed_while_in_use(shape, dtype, call)
        assert kept
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_outputs_read_on_the_current_stream(bsp, fp8):
    """Freed on the host while the current stream has yet to read them: the next call on the other stream does not get
    their memory."""
    q, run = attention(bsp, "decode", fp8)
    want = run()[0].clone()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    out, lse = run(s)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda._sleep(200_000_000)
    got = torch.empty_like(want)
    got.copy_(out)
    at = out.data_ptr()
    del out, lse
    again, _ = run(s)
    assert again.data_ptr() != at
    s.synchronize()
    again.fill_(0)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
