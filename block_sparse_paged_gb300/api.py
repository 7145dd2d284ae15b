"""Thin Python binding of the C ABI: torch tensors in, pointers to libbsp.so out.

Every step of the path runs in the library's kernels; this module only checks
shapes, dtypes and devices and passes pointers, sizes and the current stream.
"""
from __future__ import annotations

import ctypes
import math

import numpy as np
import torch

from . import _native as N

_DTYPES = {torch.bfloat16: N.BSP_DTYPE_BF16, torch.float32: N.BSP_DTYPE_F32}


def _i32_host(a) -> np.ndarray:
    if isinstance(a, torch.Tensor):
        a = a.detach().cpu().numpy()
    return np.ascontiguousarray(np.asarray(a), dtype=np.int32)


def _ptr(a: np.ndarray):
    return a.ctypes.data_as(ctypes.c_void_p)


def _stream_handle(stream) -> ctypes.c_void_p:
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _dev(t: torch.Tensor, name: str, dtype=None, device=None) -> ctypes.c_void_p:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    return ctypes.c_void_p(t.data_ptr())


def _new(stream, make):
    """make(), a tensor (or PageTables) that a call allocates for its results. It belongs to the stream that the call runs
    on, so that it takes no memory that the current stream still uses nor gives up any that `stream` still writes; and
    what the current stream does with it before it is freed comes before the memory's next use."""
    if stream is None:
        return make()
    here = torch.cuda.current_stream(stream.device)
    with torch.cuda.stream(stream):
        t = make()
    if t.is_cuda:
        t.record_stream(here)
    return t


def default_num_ctas(mode: int, device: int | None = None) -> int:
    dev = torch.cuda.current_device() if device is None else device
    out = ctypes.c_int32()
    N.check(N.load().bsp_default_num_ctas(mode, dev, ctypes.byref(out)))
    return int(out.value)


def make_problem(mode: int, num_qo_heads: int, num_kv_heads: int, head_dim: int, page_size: int,
                 causal: bool, dtype, window_left: int = -1, logits_soft_cap: float = 0.0) -> N.Problem:
    return N.Problem(mode, num_qo_heads, num_kv_heads, head_dim, page_size, int(bool(causal)), _DTYPES[dtype],
                     int(window_left), float(logits_soft_cap))


def plan_host(problem: N.Problem, capacity: N.Capacity, kv_indptr, last_page_len, qo_indptr=None,
              alpha: int = 2, beta: int = 1):
    """Plan on the host only (no device, nothing copied): returns
    (info, queue_indptr, items, merges) read back from the staging image."""
    lib = N.load()
    nbytes = lib.bsp_host_staging_size(ctypes.byref(problem), ctypes.byref(capacity))
    if nbytes == 0:
        N.check(N.BSP_ERR_INVALID_ARG)
    staging = np.zeros(nbytes, np.uint8)
    kv = _i32_host(kv_indptr)
    lp = _i32_host(last_page_len)
    qo = None if qo_indptr is None else _i32_host(qo_indptr)
    info = N.PlanInfo()
    N.check(lib.bsp_plan(ctypes.byref(problem), ctypes.byref(capacity), len(kv) - 1,
                         None if qo is None else _ptr(qo), _ptr(kv), _ptr(lp), alpha, beta,
                         _ptr(staging), None, 0, None, ctypes.byref(info)))
    return (info,) + read_plan(info, staging)


def read_plan(info: N.PlanInfo, staging: np.ndarray):
    """(queue_indptr [C+1], items, merges) from a staging image."""
    C = info.capacity.num_ctas
    q = staging[info.off_queue_indptr: info.off_queue_indptr + 4 * (C + 1)].view(np.int32).copy()
    items = staging[info.off_items: info.off_items + 64 * info.num_items].view(N.WORK_ITEM_DTYPE).copy()
    merges = staging[info.off_merges: info.off_merges + 32 * info.num_merges].view(N.MERGE_ENTRY_DTYPE).copy()
    return q, items, merges


class PagedAttention:
    """Workspace, plan and runs of block-sparse paged attention for one problem.

    mode: "decode" (one query per request, the g heads of a kv head fused into
    one tile) or "prefill" (ragged queries, 256-row tiles, tensor cores).
    max_gather_pages (prefill): pages of a K / V copy region in the workspace;
    prefills whose pages are under 8 tokens (or not a power of two) and whose
    page table fits it are gathered into it first and then read by TMA; prefills
    over an e4m3 cache with exponents convert its pages into it.
    schedule: "lpt" (the pages' plan) or "equal" (equal contiguous shares of
    the concatenated KV ranges per CTA, for batches of few, equal tiles).
    The workspace and pinned staging buffer are allocated once, for the
    given bounds; plan() may then be called once per step and run() once per
    layer, and run() can be captured in a CUDA graph. Runs of one object share
    its workspace: one at a time, on one stream or ordered by the caller.
    """

    def __init__(self, mode: str, num_qo_heads: int, num_kv_heads: int, head_dim: int, page_size: int,
                 causal: bool = False, dtype=torch.bfloat16, max_batch: int = 256,
                 max_qo_tokens: int | None = None, num_ctas: int | None = None, device=None,
                 window_left: int = -1, logits_soft_cap: float = 0.0, chunks_per_cta: int = 1,
                 max_gather_pages: int = 0, schedule: str = "lpt"):
        self.lib = N.load()
        if mode not in ("decode", "prefill"):
            raise ValueError("mode must be 'decode' or 'prefill'")
        self.mode = N.BSP_MODE_DECODE if mode == "decode" else N.BSP_MODE_PREFILL
        self.device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        self.dtype = dtype
        self.problem = make_problem(self.mode, num_qo_heads, num_kv_heads, head_dim, page_size, causal, dtype,
                                    window_left, logits_soft_cap)
        if num_ctas is None:
            num_ctas = default_num_ctas(self.mode, self.device.index)
        if max_qo_tokens is None:
            max_qo_tokens = max_batch if mode == "decode" else 65536
        if schedule not in ("lpt", "equal"):
            raise ValueError("schedule must be 'lpt' or 'equal'")
        sched = N.BSP_SCHEDULE_LPT if schedule == "lpt" else N.BSP_SCHEDULE_EQUAL_SHARES
        self.capacity = N.Capacity(max_batch, num_ctas, max_qo_tokens, chunks_per_cta, max_gather_pages, sched)
        ws_bytes = self.lib.bsp_workspace_size(ctypes.byref(self.problem), ctypes.byref(self.capacity))
        st_bytes = self.lib.bsp_host_staging_size(ctypes.byref(self.problem), ctypes.byref(self.capacity))
        if ws_bytes == 0 or st_bytes == 0:
            N.check(N.BSP_ERR_INVALID_ARG)
        self.workspace = torch.zeros(ws_bytes, dtype=torch.uint8, device=self.device)
        self.staging = torch.zeros(st_bytes, dtype=torch.uint8, pin_memory=True)
        self._copied = None  # event after the last plan copy
        self._q_tail, self._page_tail = (num_qo_heads, head_dim), (page_size, num_kv_heads, head_dim)
        self._default_scale = 1.0 / math.sqrt(head_dim)
        self.info = self._fp8_plan = self._fp8_shapes = None  # of the current plan
        self._sink_on = False  # its info points to a sink

    # ---- plan ---------------------------------------------------------------
    # Default per-position cost alpha of the LPT plan (cost of a work item =
    # alpha * query positions + beta * KV tokens). The pages' constants are
    # alpha = 2, beta = 1; a decode work item (one position) costs more than 2
    # tokens of KV on this GPU: about 64 (its setup and epilogue, measured as the
    # alpha that balanced a batch of short requests best: 59.0 -> 55.5 us).
    DEFAULT_ALPHA = {N.BSP_MODE_DECODE: 64, N.BSP_MODE_PREFILL: 2}

    def plan(self, kv_indptr, last_page_len, qo_indptr=None, alpha: int | None = None, beta: int = 1, stream=None):
        """Host plan from the request lengths; its copy is queued on `stream`.
        alpha defaults to DEFAULT_ALPHA[mode]."""
        if alpha is None:
            alpha = self.DEFAULT_ALPHA[self.mode]
        if self._copied is not None:
            self._copied.synchronize()  # the staging buffer is still the source of the previous copy
        kv = _i32_host(kv_indptr)
        lp = _i32_host(last_page_len)
        qo = None if qo_indptr is None else _i32_host(qo_indptr)
        info = N.PlanInfo()
        with torch.cuda.device(self.device):
            s = _stream_handle(stream)
            N.check(self.lib.bsp_plan(ctypes.byref(self.problem), ctypes.byref(self.capacity), len(kv) - 1,
                                      None if qo is None else _ptr(qo), _ptr(kv), _ptr(lp), alpha, beta,
                                      ctypes.c_void_p(self.staging.data_ptr()),
                                      ctypes.c_void_p(self.workspace.data_ptr()), self.workspace.numel(), s,
                                      ctypes.byref(info)))
            ev = torch.cuda.Event()
            ev.record(stream if stream is not None else torch.cuda.current_stream())
            self._copied = ev
        self.info = info
        self._fp8_plan = self._fp8_shapes = None
        self._sink_on = False
        return info

    def plan_arrays(self):
        """(queue_indptr, items, merges) of the current plan (host copy)."""
        return read_plan(self.info, self.staging.numpy())

    # ---- run ----------------------------------------------------------------
    def run(self, q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, kv_indices: torch.Tensor,
            sm_scale: float | None = None, out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
            stream=None, return_lse: bool = True, k_scale: float = 1.0, v_scale: float = 1.0,
            sink: torch.Tensor | None = None, k_exp: torch.Tensor | None = None, v_exp: torch.Tensor | None = None):
        """Attention of the planned batch. k_pages / v_pages are in the
        problem's dtype, or, for bf16 decode, torch.float8_e4m3fn pools read as
        k_scale * k_pages and v_scale * v_pages (one scale per pool), or, for bf16
        decode and prefill with head_dim 128 and any page size, such pools with one
        exponent per page and kv head: k_exp, v_exp int8 [num_pages, H_kv], value =
        code * 2^exp (the cache that append_kv writes). A prefill over such pools
        may convert the plan's pages into a bf16 copy first: in the workspace's copy
        region where max_gather_pages covers the page table, else in a temporary
        tensor of this call (a captured run that follows plans with larger tables
        needs the region: status 0x303 otherwise); a decode with pages of one or two tokens may gather the
        exponents into a temporary tensor. sink:
        float32 [H_qo] on the device, one extra softmax logit per query head
        without a value row (the attention-sink variant), or None. out and lse,
        where the call makes them, belong to `stream`."""
        if self.info is None:
            raise RuntimeError("plan() must be called before run()")
        if k_exp is not None or v_exp is not None:
            return self._run_fp8_block(q, k_pages, v_pages, k_exp, v_exp, kv_indices, sm_scale, out, lse, stream,
                                       return_lse, k_scale, v_scale, sink)
        P = self.problem
        D = P.head_dim
        if q.dim() != 3 or q.shape[1] != P.num_qo_heads or q.shape[2] != D:
            raise ValueError(f"q must be [n_tokens, {P.num_qo_heads}, {D}]")
        if k_pages.dim() != 4 or k_pages.shape[1:] != (P.page_size, P.num_kv_heads, D) or v_pages.shape != k_pages.shape:
            raise ValueError(f"k_pages / v_pages must be [num_pages, {P.page_size}, {P.num_kv_heads}, {D}]")
        if sm_scale is None:
            sm_scale = 1.0 / math.sqrt(D)
        if out is None:
            out = _new(stream, lambda: torch.empty_like(q))
        if lse is None and return_lse:
            lse = _new(stream, lambda: torch.empty(q.shape[:2], dtype=torch.float32, device=q.device))
        dev = self.device
        fp8 = k_pages.dtype == torch.float8_e4m3fn
        if fp8 and (self.mode != N.BSP_MODE_DECODE or self.dtype != torch.bfloat16):
            raise ValueError("e4m3 KV pools are read by the bf16 decode run only")
        kv_dt = torch.float8_e4m3fn if fp8 else self.dtype
        if not fp8 and (k_scale != 1.0 or v_scale != 1.0):
            raise ValueError("k_scale / v_scale apply to e4m3 KV pools only")
        args = [ctypes.byref(self.info), _dev(q, "q", self.dtype, dev), _dev(k_pages, "k_pages", kv_dt, dev),
                _dev(v_pages, "v_pages", kv_dt, dev), _dev(kv_indices, "kv_indices", torch.int32, dev)
                if kv_indices.numel() else None]
        tail = [ctypes.c_float(sm_scale), _dev(out, "out", self.dtype, dev),
                None if lse is None else _dev(lse, "lse", torch.float32, dev),
                ctypes.c_void_p(self.workspace.data_ptr())]
        self._set_sink(sink)
        with torch.cuda.device(dev):
            s = _stream_handle(stream)
            if fp8:
                N.check(self.lib.bsp_decode_run_fp8(*args, k_pages.shape[0], tail[0], ctypes.c_float(k_scale),
                                                    ctypes.c_float(v_scale), *tail[1:], s))
            elif self.mode == N.BSP_MODE_DECODE:
                N.check(self.lib.bsp_decode_run(*args, k_pages.shape[0], *tail, s))
            else:
                N.check(self.lib.bsp_prefill_run(*args, k_pages.shape[0], *tail, s))
        return (out, lse) if return_lse else out

    def _run_fp8_block(self, q, k_pages, v_pages, k_exp, v_exp, kv_indices, sm_scale, out, lse, stream, return_lse,
                       k_scale, v_scale, sink):
        """run() over an e4m3 cache with one exponent per page and kv head. (A short step's time is this function's:
        what depends on the plan and on shapes alone is looked at once per plan.)"""
        dev, f8, i8 = self.device, torch.float8_e4m3fn, torch.int8
        if k_exp is None or v_exp is None:
            raise ValueError("k_exp and v_exp are given together")
        if k_scale != 1.0 or v_scale != 1.0:
            raise ValueError("k_scale / v_scale do not apply to pools with exponents")
        if self.dtype is not torch.bfloat16:
            raise ValueError("pools with exponents are read by bfloat16 problems")
        q_shape, pool = q.shape, k_pages.shape
        shapes = (q_shape, pool, v_pages.shape, k_exp.shape, v_exp.shape, kv_indices.shape)
        if shapes != self._fp8_shapes:
            self._check_fp8_shapes(*shapes)
            self._fp8_shapes = shapes
        ref, fn, region, nbytes, ws = self._fp8_plan or self._look_at_fp8_plan()
        q_p = _addr(q, "q", torch.bfloat16, dev)
        if out is None:
            out = _new(stream, lambda: torch.empty_like(q))
            out_p = out.data_ptr()
        else:
            if out.shape != q_shape:
                raise ValueError("out must have the shape of q")
            out_p = _addr(out, "out", torch.bfloat16, dev)
        lse_p = None
        if lse is not None:
            if lse.shape != q_shape[:2]:
                raise ValueError("lse must be [n_tokens, H_qo]")
            lse_p = _addr(lse, "lse", torch.float32, dev)
        elif return_lse:
            lse = _new(stream, lambda: torch.empty(q_shape[:2], dtype=torch.float32, device=dev))
            lse_p = lse.data_ptr()
        if sm_scale is None:
            sm_scale = self._default_scale
        if sink is not None or self._sink_on:
            self._set_sink(sink)
        copy = None
        if nbytes and region is None:  # scratch of this run alone: the plan's exponents, or a bf16 copy of its pages
            if stream is None:
                copy = torch.empty(nbytes, dtype=torch.uint8, device=dev)
            else:
                with torch.cuda.stream(stream):
                    copy = torch.empty(nbytes, dtype=torch.uint8, device=dev)
            region = copy.data_ptr()
        _call(dev, stream, fn, ref, q_p, _addr(k_pages, "k_pages", f8, dev), _addr(v_pages, "v_pages", f8, dev),
              _addr(k_exp, "k_exp", i8, dev), _addr(v_exp, "v_exp", i8, dev),
              _addr(kv_indices, "kv_indices", torch.int32, dev) or None, pool[0], sm_scale, out_p, lse_p, region, nbytes, ws)
        return (out, lse) if return_lse else out

    def _check_fp8_shapes(self, q, k_pages, v_pages, k_exp, v_exp, kv_indices):
        info = self.info
        if q[1:] != self._q_tail or q[0] < info.num_qo_tokens:
            raise ValueError(f"q must be [n_tokens, {self._q_tail[0]}, {self._q_tail[1]}] with the plan's tokens")
        if k_pages[1:] != self._page_tail or v_pages != k_pages:
            raise ValueError("k_pages / v_pages must be [num_pages, %d, %d, %d]" % self._page_tail)
        if k_exp != (k_pages[0], k_pages[2]) or v_exp != k_exp:
            raise ValueError(f"k_exp / v_exp must be [{k_pages[0]}, {k_pages[2]}]")
        if len(kv_indices) != 1 or kv_indices[0] < info.num_table_pages:
            raise ValueError(f"kv_indices must hold the plan's {info.num_table_pages} pages")

    def _look_at_fp8_plan(self):
        """(plan info reference, entry, region in the workspace or None, region bytes, workspace) of the current plan."""
        info, lib, ws, ref = self.info, self.lib, self.workspace.data_ptr(), ctypes.byref(self.info)
        region = None
        if self.mode == N.BSP_MODE_DECODE:
            fn, nbytes = lib.bsp_decode_run_fp8_block, lib.bsp_decode_fp8_region_size(ref)
        else:
            fn, nbytes = lib.bsp_prefill_run_fp8_block, lib.bsp_prefill_fp8_region_size(ref)
            if nbytes and self.capacity.max_gather_pages >= info.num_table_pages:
                region, nbytes = ws + info.off_gather, 2 * info.gather_pool_bytes  # the workspace's copy region
        self._fp8_plan = (ref, fn, region, nbytes, ws)
        return self._fp8_plan

    def _set_sink(self, sink):
        self._sink_on = sink is not None
        if sink is None:
            self.info.problem.sink = None
            return
        if sink.dim() != 1 or sink.shape[0] != self.problem.num_qo_heads:
            raise ValueError(f"sink must be [{self.problem.num_qo_heads}]")
        self.info.problem.sink = _dev(sink, "sink", torch.float32, self.device).value
        self._sink_ref = sink  # the kernel reads it during the run

    def run_stages(self, q, k_pages, v_pages, kv_indices, sm_scale, out, lse, stream=None, events=None):
        """The run as its launches on `stream`: the attention kernel, then for
        prefill the merge of partials (decode merges inside its kernel);
        `events` = (e0, e1, e2) are recorded before, between and after them when
        given. out and lse must be preallocated."""
        dev = self.device
        with torch.cuda.device(dev):
            st = stream if stream is not None else torch.cuda.current_stream()
            s = ctypes.c_void_p(st.cuda_stream)
            ws = ctypes.c_void_p(self.workspace.data_ptr())
            o_p = _dev(out, "out", self.dtype, dev)
            l_p = None if lse is None else _dev(lse, "lse", torch.float32, dev)
            self._set_sink(None)
            if events:
                events[0].record(st)
            N.check(self.lib.bsp_run_attention(ctypes.byref(self.info), _dev(q, "q", self.dtype, dev),
                                               _dev(k_pages, "k_pages", self.dtype, dev),
                                               _dev(v_pages, "v_pages", self.dtype, dev),
                                               _dev(kv_indices, "kv_indices", torch.int32, dev), k_pages.shape[0],
                                               ctypes.c_float(sm_scale), o_p, l_p, ws, s))
            if events:
                events[1].record(st)
            if self.mode == N.BSP_MODE_PREFILL:  # decode merges split outputs inside its kernel
                N.check(self.lib.bsp_run_merge_partials(ctypes.byref(self.info), o_p, l_p, ws, s))
            if events:
                events[2].record(st)
        return out, lse

    def check_device_error(self, stream=None) -> int:
        word = ctypes.c_int32()
        with torch.cuda.device(self.device):
            N.check(self.lib.bsp_check_device_error(ctypes.byref(self.info), ctypes.c_void_p(self.workspace.data_ptr()),
                                                    _stream_handle(stream), ctypes.byref(word)))
        return int(word.value)


def merge_state(o_a: torch.Tensor, lse_a: torch.Tensor, o_b: torch.Tensor, lse_b: torch.Tensor,
                out: torch.Tensor | None = None, lse_out: torch.Tensor | None = None, stream=None):
    """Merge two sets of attention states O [n, H, D], LSE [n, H] (float32)."""
    if o_a.shape != o_b.shape or o_a.dim() != 3 or lse_a.shape != o_a.shape[:2] or lse_b.shape != lse_a.shape:
        raise ValueError("o_a, o_b must be [n, H, D] and lse_a, lse_b [n, H]")
    dt = o_a.dtype
    if dt not in _DTYPES:
        raise ValueError("dtype must be bfloat16 or float32")
    if out is None:
        out = _new(stream, lambda: torch.empty_like(o_a))
    if lse_out is None:
        lse_out = _new(stream, lambda: torch.empty_like(lse_a))
    n, H, D = o_a.shape
    lib = N.load()
    with torch.cuda.device(o_a.device):
        N.check(lib.bsp_merge_state(_dev(o_a, "o_a", dt), _dev(lse_a, "lse_a", torch.float32), _dev(o_b, "o_b", dt),
                                    _dev(lse_b, "lse_b", torch.float32), _dev(out, "out", dt),
                                    _dev(lse_out, "lse_out", torch.float32), n, H, D, _DTYPES[dt],
                                    _stream_handle(stream)))
    return out, lse_out


def _addr(t: torch.Tensor, name: str, dtype, dev: torch.device) -> int:
    """Address of a contiguous tensor of `dtype` on `dev`; _dev's errors otherwise (short calls: checked once, in the
    order of what is cheap to ask)."""
    if t.dtype is dtype and t.is_contiguous() and t.device == dev:
        return t.data_ptr()
    return _dev(t, name, dtype, dev).value


def _call(dev: torch.device, stream, fn, *args):
    """fn(*args, stream handle) with `dev` current, on `stream` or dev's current stream."""
    # (the handle of torch.cuda.current_stream(dev), without making the object)
    handle = stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(dev.index)
    if dev.index != torch._C._cuda_getDevice():
        with torch.cuda.device(dev):
            rc = fn(*args, handle)
    else:
        rc = fn(*args, handle)
    if rc != N.BSP_OK:
        N.check(rc)


class PageTables:
    """What build_page_tables writes, for up to the given sizes: int32 kv_indptr
    [batch + 1], last_page_len [batch], kv_indices [max_table_pages], qo_indptr
    [batch + 1], positions [max_new_tokens], counts [4] (table pages, new tokens,
    pages taken, error bits BSP_TABLES_*) and int64 slot_map [max_new_tokens]. The
    int32 arrays are parts of one buffer; to be kept and passed as `out` every step."""
    is_cuda = True
    _fields = ("kv_indptr", "last_page_len", "kv_indices", "qo_indptr", "slot_map", "positions", "counts")

    def __init__(self, batch: int, max_table_pages: int, max_new_tokens: int, device=None):
        if min(batch, max_table_pages, max_new_tokens) < 0:
            raise ValueError("sizes must not be negative")
        dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        self.sizes = (batch, max_table_pages, max_new_tokens)
        parts = [("kv_indices", max_table_pages), ("positions", max_new_tokens), ("kv_indptr", batch + 1),
                 ("qo_indptr", batch + 1), ("last_page_len", batch), ("counts", 4)]
        at, offsets = 0, {}
        for f, n in parts:  # every part 16-byte aligned
            offsets[f] = at
            at += (n + 3) // 4 * 4
        self._ints = torch.empty(at, dtype=torch.int32, device=dev)
        self.slot_map = torch.empty(max_new_tokens, dtype=torch.int64, device=dev)
        for f, n in parts:
            setattr(self, f, self._ints[offsets[f]:offsets[f] + n])
        self._offsets = tuple(4 * offsets[f] for f in ("kv_indptr", "last_page_len", "kv_indices", "qo_indptr",
                                                       "positions", "counts"))
        self.device = self._ints.device

    def record_stream(self, stream) -> None:
        """As of a tensor: memory that `stream` uses too."""
        self._ints.record_stream(stream)
        self.slot_map.record_stream(stream)

    @classmethod
    def empty(cls, batch: int, max_table_pages: int, max_new_tokens: int, device=None) -> "PageTables":
        """Buffers of these sizes, not yet written."""
        return cls(batch, max_table_pages, max_new_tokens, device)


def build_page_tables(cached_lens: torch.Tensor, new_lens: torch.Tensor, free_pages: torch.Tensor,
                      num_free: torch.Tensor, block_table: torch.Tensor, page_size: int, max_table_pages: int,
                      max_new_tokens: int, out: PageTables | None = None, stream=None) -> PageTables:
    """Page table (CSR), slots and positions of one step from the request lengths
    on the device (bsp_build_page_tables).

    cached_lens, new_lens: int32 [B], tokens in the cache and tokens added by this
    step. block_table: int32 [B, width], rows of adjacent entries; the rows' pages
    for the cached tokens are read, the pages that the new tokens need are taken
    from free_pages (int32, the first num_free [1] of them) and written.
    max_table_pages / max_new_tokens: sizes of kv_indices and of slot_map and
    positions, whose tails are filled with 0, -1 and 0. Nothing is read back: whether
    all fitted stands in counts[3]."""
    if block_table.dim() != 2:
        raise ValueError("block_table must be [B, width] with adjacent entries in a row")
    B, width = block_table.shape
    stride, step = block_table.stride()
    if step != 1 and B > 0 and width > 1:
        raise ValueError("block_table must be [B, width] with adjacent entries in a row")
    dev = block_table.device
    if not block_table.is_cuda or block_table.dtype is not torch.int32:
        raise ValueError("block_table must be a CUDA tensor of torch.int32")
    if cached_lens.shape != (B,) or new_lens.shape != (B,):
        raise ValueError(f"cached_lens and new_lens must be [{B}]")
    if free_pages.dim() != 1 or num_free.numel() != 1:
        raise ValueError("free_pages must be one-dimensional and num_free hold one value")
    if out is None:
        out = _new(stream, lambda: PageTables(B, max_table_pages, max_new_tokens, dev))
    elif out.sizes != (B, max_table_pages, max_new_tokens) or out.device != dev:
        raise ValueError(f"out is for {out.sizes} (batch, pages, tokens) on {out.device}")
    if B <= 1:
        stride = max(width, stride)
    i32 = torch.int32
    o = out._ints.data_ptr()
    kv_indptr, last, indices, qo_indptr, pos, counts = out._offsets
    _call(dev, stream, N.load().bsp_build_page_tables, B, page_size, _addr(cached_lens, "cached_lens", i32, dev),
          _addr(new_lens, "new_lens", i32, dev), _addr(free_pages, "free_pages", i32, dev), free_pages.shape[0],
          _addr(num_free, "num_free", i32, dev), block_table.data_ptr(), stride, width, o + kv_indptr, o + last,
          o + indices, max_table_pages, o + qo_indptr, out.slot_map.data_ptr(), o + pos, max_new_tokens, o + counts)
    return out


def append_kv(k: torch.Tensor, v: torch.Tensor, slot_map: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
              k_exp: torch.Tensor, v_exp: torch.Tensor, stream=None) -> None:
    """Quantise new keys and values into the e4m3 cache, in place (bsp_append_kv_fp8).

    k, v: [n, H_kv, 128] bfloat16 or float32, slices of larger tensors allowed (the
    values of a row adjacent, 16-byte aligned rows). slot_map: int64 [n], page *
    page_size + place, as build_page_tables gives it; tokens with a slot outside the
    pool are skipped. k_pages, v_pages: float8_e4m3fn [num_pages, page_size, H_kv,
    128]; k_exp, v_exp: int8 [num_pages, H_kv], value = code * 2^exp."""
    pool, shape, dtype, dev = k_pages.shape, k.shape, k.dtype, k_pages.device
    if len(pool) != 4 or v_pages.shape != pool:
        raise ValueError("k_pages / v_pages must be [num_pages, page_size, H_kv, D]")
    P, ps, H, D = pool
    if len(shape) != 3 or shape[1] != H or shape[2] != D or v.shape != shape or v.dtype is not dtype or dtype not in _DTYPES:
        raise ValueError(f"k and v must be [n, {H}, {D}] in bfloat16 or float32, of one type")
    n, ks, vs = shape[0], k.stride(), v.stride()
    if ks[2] != 1 or vs[2] != 1:
        raise ValueError("the values of a row of k and v must be adjacent")
    if slot_map.dim() != 1 or slot_map.numel() != n:
        raise ValueError(f"slot_map must be [{n}]")
    if k_exp.shape != (P, H) or v_exp.shape != (P, H):
        raise ValueError(f"k_exp / v_exp must be [{P}, {H}]")
    if not k.is_cuda or k.device != dev or v.device != dev:
        raise ValueError(f"k and v must be CUDA tensors on {dev}")
    f8, i8 = torch.float8_e4m3fn, torch.int8
    # a dimension of size 1 is never stepped over: its stride says nothing
    if n == 1:
        ks, vs = (0,) + ks[1:], (0,) + vs[1:]
    if H == 1:
        ks, vs = (ks[0], 0), (vs[0], 0)
    _call(dev, stream, N.load().bsp_append_kv_fp8, k.data_ptr(), v.data_ptr(), ks[0], ks[1], vs[0], vs[1],
          _DTYPES[dtype], n, _addr(slot_map, "slot_map", torch.int64, dev), _addr(k_pages, "k_pages", f8, dev),
          _addr(v_pages, "v_pages", f8, dev), _addr(k_exp, "k_exp", i8, dev), _addr(v_exp, "v_exp", i8, dev), P, ps, H, D)
