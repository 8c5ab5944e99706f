"""The paged key-value cache: page tables, stores, and attention of one new token.

    pages = lb.PageTable(table, page_size, num_pages, max_tokens)   # table: (max_requests, max_pages) int32
    pages.append(past, fresh, free_pages)                           # one step: new tokens' pages and slots
    lb.paged_store(k, v, k_cache, v_cache, pages.slots)             # (tokens, kv_heads, head_dim)
    attend = lb.PagedAttention(max_batch, q_heads, kv_heads, head_dim, torch.bfloat16)
    out, lse = attend(q, k_cache, v_cache, table, pages.lens)       # q: (batch, q_heads, head_dim)

Caches are (num_pages, page_size, kv_heads, head_dim) tensors or views of any
layout whose last dimension is contiguous (a cache kept head by head is passed
as its transposed view).  Argument marshalling only; include/spmv.h
(spmv_pages_append, spmv_paged_store, spmv_paged_attention) has the contract.
"""
from __future__ import annotations

import ctypes

import torch

from . import _launch, check, lib

__all__ = ["PageTable", "PagedAttention", "paged_store"]


class PageTable:
    """The page table of a cache of ``num_pages`` pages of ``page_size``
    tokens.  ``table`` (max_requests, max_pages), int32, is the caller's and
    is extended in place.  ``append`` fills, for the requests of one step,
    ``token_ptr`` (requests + 1), ``lens`` (requests), ``slots`` and
    ``positions`` (max_tokens) and ``taken`` (1), and adds its flags to
    ``status`` (1).  Keep the object until its calls have run."""

    def __init__(self, table, page_size: int, num_pages: int, max_tokens: int):
        if table.dtype != torch.int32 or not table.is_cuda or table.dim() != 2:
            raise TypeError("table must be a two-dimensional CUDA int32 tensor")
        self._L, self.table, self.device = lib(), table, table.device
        self.page_size, self.num_pages, self.max_tokens = int(page_size), int(num_pages), int(max_tokens)
        self.max_requests, self.max_pages = table.shape
        self._ld = _launch.rows("table", table, table.shape, torch.int32, self.device)
        self._table_ptr = table.data_ptr()
        size = ctypes.c_size_t()
        check(self._L.spmv_pages_workspace(self.max_requests, ctypes.byref(size)), "spmv_pages_workspace")
        int32 = dict(dtype=torch.int32, device=self.device)
        self._token_ptr = torch.empty(self.max_requests + 1, **int32)
        self._lens = torch.empty(self.max_requests, **int32)
        self.slots, self.positions = (torch.empty(self.max_tokens, **int32) for _ in range(2))
        self.taken, self.status = torch.zeros(1, **int32), torch.zeros(1, **int32)
        self._workspace = torch.empty(size.value, dtype=torch.uint8, device=self.device)
        self._outputs = (self._token_ptr.data_ptr(), self._lens.data_ptr(), self.slots.data_ptr(),
                         self.positions.data_ptr(), self.taken.data_ptr(), self.status.data_ptr(),
                         self._workspace.data_ptr(), size.value)
        self.token_ptr = self.lens = None
        self._requests = None
        _launch.settle(self.device)

    def append(self, past, fresh, free_pages, stream=None) -> "PageTable":
        """Add ``fresh[r]`` tokens to request r, which holds ``past[r]``
        (both int32, one entry per request of the step, in the table's row
        order); new pages come from ``free_pages`` (int32) in its order.
        ``past`` must not be ``lens`` itself: a step's lens is copied before
        it is the next step's past."""
        d, n, free = self.device, past.numel(), free_pages.numel()
        if n > self.max_requests:
            raise ValueError(f"{n} requests, but the table has {self.max_requests} rows")
        if fresh.numel() != n:
            raise ValueError("past and fresh differ in length")
        past_ptr = _launch.vector("past", past, n, torch.int32, d)
        fresh_ptr = _launch.vector("fresh", fresh, n, torch.int32, d)
        free_ptr = _launch.vector("free_pages", free_pages, free, torch.int32, d)
        _launch.call(self._L.spmv_pages_append, "spmv_pages_append", d, n, past_ptr, fresh_ptr, self.page_size,
                     self.num_pages, free_ptr, free, self._table_ptr, self._ld, self.max_pages, self.max_tokens,
                     *self._outputs, _launch.handle(stream, d))
        if n != self._requests:
            self.token_ptr, self.lens, self._requests = self._token_ptr[:n + 1], self._lens[:n], n
        return self


def _cache_strides(name, cache, heads, dim, dtype, device):
    if cache.dtype != dtype or cache.device != device:
        raise TypeError(f"{name} must be a {dtype} tensor on {device}, got {cache.dtype} on {cache.device}")
    if cache.dim() != 4 or cache.shape[2] != heads or cache.shape[3] != dim:
        raise ValueError(f"{name} must be (pages, page_size, {heads}, {dim}), got {tuple(cache.shape)}")
    strides = cache.stride()
    if strides[3] != 1:
        raise ValueError(f"{name} must have a contiguous last dimension")
    return strides


_I64x2, _I64x3 = ctypes.c_int64 * 2, ctypes.c_int64 * 3

_store_seen = {}  # the layouts that were checked last, and what the checks gave


def _check_store(k, v, k_cache, v_cache):
    d, dtype = k.device, k.dtype
    if not k.is_cuda:
        raise TypeError("k must be a CUDA tensor")
    if k.dim() != 3 or v.shape != k.shape:
        raise ValueError("k and v must be (tokens, kv_heads, head_dim)")
    if v.dtype != dtype or v.device != d:
        raise TypeError("k and v differ in type or device")
    tokens, heads, dim = k.shape
    ks, vs = k.stride(), v.stride()
    if (ks[2] != 1 or vs[2] != 1) and dim > 1:
        raise ValueError("k and v must have a contiguous last dimension")
    kc = _cache_strides("k_cache", k_cache, heads, dim, dtype, d)
    vc = _cache_strides("v_cache", v_cache, heads, dim, dtype, d)
    if k_cache.shape != v_cache.shape:
        raise ValueError("k_cache and v_cache differ in shape")
    return (d, (tokens, heads, dim, _launch.elem(dtype)), tuple(k_cache.shape[:2]),
            _I64x2(*ks[:2]), _I64x2(*vs[:2]), _I64x3(*kc[:3]), _I64x3(*vc[:3]))


def paged_store(k, v, k_cache, v_cache, slots, stream=None) -> None:
    """Write token i's keys and values (k, v: (tokens, kv_heads, head_dim),
    contiguous in the last dimension) into slot ``slots[i]`` (int32) of the
    caches; slots outside the caches (-1: padding) are skipped.  For serving:
    no gradient flows through the caches."""
    like = (k.shape, k.stride(), k.dtype, k.device, v.shape, v.stride(), v.dtype, v.device,
            k_cache.shape, k_cache.stride(), k_cache.dtype, k_cache.device,
            v_cache.shape, v_cache.stride(), v_cache.dtype, v_cache.device)
    known = _store_seen.get("last")
    if known is None or known[0] != like:
        known = like, _check_store(k, v, k_cache, v_cache)
        _store_seen["last"] = known
    d, sizes, pages, ks, vs, kc, vc = known[1]
    at = _launch.vector("slots", slots, sizes[0], torch.int32, d)
    _launch.call(lib().spmv_paged_store, "spmv_paged_store", d, *sizes, at, *pages, k.data_ptr(), ks, v.data_ptr(), vs,
                 k_cache.data_ptr(), kc, v_cache.data_ptr(), vc, _launch.handle(stream, d))


class PagedAttentionArgs(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("q_heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32), ("num_pages", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("elem", ctypes.c_int32), ("scale", ctypes.c_float),
                ("reserved", ctypes.c_int32), ("q_stride", _I64x2), ("k_stride", _I64x3), ("v_stride", _I64x3),
                ("out_stride", _I64x2), ("table_stride", ctypes.c_int64), ("q", ctypes.c_void_p),
                ("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("lens", ctypes.c_void_p), ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t), ("status", ctypes.c_void_p)]


class PagedAttention:
    """Attention of one new token for each of up to ``max_batch`` requests.
    Keeps the workspace that joins requests cut between blocks: calls that may
    overlap on the GPU (two streams) need objects of their own, and an object
    is kept until its calls have run."""

    def __init__(self, max_batch: int, q_heads: int, kv_heads: int, head_dim: int, dtype, device="cuda"):
        self._L, self.device, self.dtype = lib(), _launch.cuda_device(device), dtype
        self._args = a = PagedAttentionArgs()
        a.elem = _launch.elem(dtype)
        self.max_batch = int(max_batch)
        self.q_heads, self.kv_heads, self.head_dim = int(q_heads), int(kv_heads), int(head_dim)
        a.q_heads, a.kv_heads, a.head_dim = self.q_heads, self.kv_heads, self.head_dim
        size = ctypes.c_size_t()
        with torch.cuda.device(self.device):
            check(self._L.spmv_paged_attention_workspace(self.max_batch, self.q_heads, self.kv_heads, self.head_dim,
                                                         a.elem, ctypes.byref(size)), "spmv_paged_attention_workspace")
        self._workspace = torch.empty(size.value, dtype=torch.uint8, device=self.device)
        self._workspace[:4096].zero_()
        self._status = torch.zeros(1, dtype=torch.int32, device=self.device)
        # the inputs' layouts that were checked last, and the outputs' shapes for them; whether the arguments have
        # the strides of a new output
        self._like = self._shape = None
        self._dense, self._scale, self._args_ref = False, self.head_dim ** -0.5, ctypes.byref(a)
        a.workspace, a.workspace_bytes, a.status = (self._workspace.data_ptr(), size.value,
                                                    self._status.data_ptr())
        _launch.settle(self.device)

    def __call__(self, q, k_cache, v_cache, table, lens, scale=None, out=None, lse=None, stream=None):
        """(out, lse) of q (batch, q_heads, head_dim) over the first
        ``lens[b]`` (int32) positions of each request, whose pages are row b
        of ``table`` (int32).  ``scale``: head_dim ** -0.5 if None.  It has no
        derivative."""
        if _launch.tracked(q, k_cache, v_cache, out):
            _launch.no_outputs_given("PagedAttention", out, lse)
            with _launch.on(stream, self.device):
                return _launch.NoDerivative.apply("PagedAttention", lambda: self._attend(q, k_cache, v_cache, table, lens, scale),
                                                  q, k_cache, v_cache)
        return self._attend(q, k_cache, v_cache, table, lens, scale, out, lse, stream)

    def _attend(self, q, k_cache, v_cache, table, lens, scale=None, out=None, lse=None, stream=None):
        d, a = self.device, self._args
        like = (q.shape, q.stride(), q.dtype, q.device, k_cache.shape, k_cache.stride(), k_cache.dtype, k_cache.device,
                v_cache.shape, v_cache.stride(), v_cache.dtype, v_cache.device, table.shape, table.stride(), table.dtype,
                table.device, lens.shape, lens.stride(), lens.dtype, lens.device)
        if like != self._like:
            self._like = None
            self._check(q, k_cache, v_cache, table, lens)
            self._like, self._shape, self._dense = like, (q.shape, q.shape[:2]), False
        shape, heads = self._shape
        if out is not None:
            if out.dtype != self.dtype or out.device != d or out.shape != shape or out.stride(2) != 1:
                raise ValueError(f"out must be a {self.dtype} tensor of shape {tuple(shape)} on {d}, contiguous in its last "
                                 "dimension")
            a.out_stride[:] = out.stride()[:2]
            self._dense = False
        else:
            out = _launch.empty(stream, d, shape, self.dtype)
            if not self._dense:
                a.out_stride[:] = out.stride()[:2]
                self._dense = True
        if lse is None:
            lse = _launch.empty(stream, d, heads, torch.float32)
        elif lse.dtype != torch.float32 or lse.device != d or lse.shape != heads or not lse.is_contiguous():
            raise ValueError(f"lse must be a contiguous float32 tensor of shape {tuple(heads)} on {d}")
        a.scale = self._scale if scale is None else scale
        a.q, a.k_cache, a.v_cache = q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr()
        a.table, a.lens, a.out, a.lse = table.data_ptr(), lens.data_ptr(), out.data_ptr(), lse.data_ptr()
        _launch.call(self._L.spmv_paged_attention, "spmv_paged_attention", d, self._args_ref,
                     _launch.handle(stream, d))
        return out, lse

    def _check(self, q, k_cache, v_cache, table, lens):
        """Checks the inputs' layouts and puts them into the arguments."""
        d, dtype, dim, hq, a = self.device, self.dtype, self.head_dim, self.q_heads, self._args
        if q.dtype != dtype or q.device != d:
            raise TypeError(f"q must be a {dtype} tensor on {d}, got {q.dtype} on {q.device}")
        if q.dim() != 3 or q.shape[1:] != (hq, dim) or q.shape[0] > self.max_batch:
            raise ValueError(f"q must be (batch <= {self.max_batch}, {hq}, {dim}), got {tuple(q.shape)}")
        batch, qs = q.shape[0], q.stride()
        if qs[2] != 1:
            raise ValueError("q must have a contiguous last dimension")
        ks = _cache_strides("k_cache", k_cache, self.kv_heads, dim, dtype, d)
        vs = _cache_strides("v_cache", v_cache, self.kv_heads, dim, dtype, d)
        if k_cache.shape != v_cache.shape:
            raise ValueError("k_cache and v_cache differ in shape")
        if table.dim() != 2 or table.shape[0] < batch:
            raise ValueError("table must have a row for each request")
        a.table_stride = _launch.rows("table", table, table.shape, torch.int32, d)
        _launch.vector("lens", lens, batch, torch.int32, d)
        a.batch = batch
        a.num_pages, a.page_size = k_cache.shape[:2]
        a.max_pages = table.shape[1]
        a.q_stride[:], a.k_stride[:], a.v_stride[:] = qs[:2], ks[:3], vs[:3]

    def device_status(self) -> int:
        """Flags of the calls so far (0 = none); waits for the device.  Bit 0:
        a page outside the cache; bit 1: a length outside its table row."""
        torch.cuda.synchronize(self.device)
        return int(self._status.item())
