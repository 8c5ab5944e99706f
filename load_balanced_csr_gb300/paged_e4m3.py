"""The paged cache in 8 bits: quantising stores, reading back, and attention of one new token.

    kc, vc = (torch.empty(pages, page_size, kv_heads, head_dim, dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2))
    ks, vs = (torch.empty(pages, page_size // block, kv_heads, device="cuda") for _ in range(2))  # a scale per block and head
    lb.paged_store_e4m3(k, v, kc, vc, ks, vs, pages.slots)           # (tokens, kv_heads, head_dim), quantised as it is written
    k, v = lb.paged_load(kc, vc, pages.table, kv_ptr, tokens, ks, vs, dtype=torch.bfloat16)
    attend = lb.PagedAttentionE4M3(max_batch, q_heads, kv_heads, head_dim, torch.bfloat16)
    out, lse = attend(q, kc, vc, ks, vs, pages.table, pages.lens)    # q: (batch, q_heads, head_dim)

Caches are float8_e4m3fn tensors or views of any layout whose last dimension is
contiguous, scales float32 tensors of any strides.  An element stands for its
code times the scale of its block of ``page_size // scales.shape[1]`` positions.
``paged_load`` reads caches of whole elements too.  Argument marshalling only;
include/spmv.h (spmv_paged_cache_t, spmv_paged_store_e4m3, spmv_paged_load,
spmv_paged_attention_e4m3) has the contract.
"""
from __future__ import annotations

import ctypes

import torch

from . import _launch, check, lib
from .paged import PagedAttention, _cache_strides, _I64x2, _I64x3

__all__ = ["PagedAttentionE4M3", "paged_load", "paged_store_e4m3"]

CODES = torch.float8_e4m3fn


class PagedCacheArgs(ctypes.Structure):
    _fields_ = [("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("block", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("k_stride", _I64x3), ("v_stride", _I64x3), ("k_scale_stride", _I64x3),
                ("v_scale_stride", _I64x3), ("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p),
                ("k_scales", ctypes.c_void_p), ("v_scales", ctypes.c_void_p)]


def _layout(t):
    return None if t is None else (t.shape, t.stride(), t.dtype, t.device)


def _scale_block(k_cache, k_scales, v_scales, device):
    """Checks the scales of a cache of codes and returns a block's positions."""
    pages, page, heads, _ = k_cache.shape
    for name, s in (("k_scales", k_scales), ("v_scales", v_scales)):
        if s is None or s.dtype != torch.float32 or s.device != device:
            raise TypeError(f"{name} must be a float32 tensor on {device}")
        if s.dim() != 3 or s.shape[0] != pages or s.shape[2] != heads or not 1 <= s.shape[1] <= page or page % s.shape[1]:
            raise ValueError(f"{name} must be ({pages}, a divisor of {page}, {heads}), got {tuple(s.shape)}")
    if k_scales.shape != v_scales.shape:
        raise ValueError("k_scales and v_scales differ in shape")
    return page // k_scales.shape[1]


def _cache_args(k_cache, v_cache, k_scales, v_scales, heads, dim, dtype, device):
    """The checked layout of a cache, without its addresses."""
    ks = _cache_strides("k_cache", k_cache, heads, dim, dtype, device)
    vs = _cache_strides("v_cache", v_cache, heads, dim, dtype, device)
    if k_cache.shape != v_cache.shape:
        raise ValueError("k_cache and v_cache differ in shape")
    _launch.counts(*k_cache.shape)
    a = PagedCacheArgs()
    a.num_pages, a.page_size = k_cache.shape[:2]
    a.k_stride[:], a.v_stride[:] = ks[:3], vs[:3]
    if dtype == CODES:
        if a.page_size < 1:
            raise ValueError("page_size must be at least 1")
        a.block = _scale_block(k_cache, k_scales, v_scales, device)
        a.k_scale_stride[:], a.v_scale_stride[:] = k_scales.stride(), v_scales.stride()
    return a


def _with_addresses(like, k_cache, v_cache, k_scales, v_scales):
    """A layout with its addresses: a structure of its own, since host threads may call at once."""
    a = PagedCacheArgs()
    ctypes.memmove(ctypes.byref(a), ctypes.byref(like), ctypes.sizeof(a))
    a.k_cache, a.v_cache = k_cache.data_ptr(), v_cache.data_ptr()
    if a.block:
        a.k_scales, a.v_scales = k_scales.data_ptr(), v_scales.data_ptr()
    return a


def _token_strides(name, t, shape, dtype, device):
    if t.dtype != dtype or t.device != device:
        raise TypeError(f"{name} must be a {dtype} tensor on {device}, got {t.dtype} on {t.device}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    strides = t.stride()
    if strides[2] != 1 and shape[2] > 1:
        raise ValueError(f"{name} must have a contiguous last dimension")
    return _I64x2(*strides[:2])


_seen = {}  # the layouts that were checked last, and what the checks gave


def _check_store(k, v, k_cache, v_cache, k_scales, v_scales):
    d, dtype = k.device, k.dtype
    if not k.is_cuda:
        raise TypeError("k must be a CUDA tensor")
    if k.dim() != 3:
        raise ValueError("k and v must be (tokens, kv_heads, head_dim)")
    tokens, heads, dim = k.shape
    if k_cache.dtype != CODES:
        raise TypeError(f"k_cache must be a {CODES} tensor, got {k_cache.dtype}")
    _launch.counts(tokens)
    return (d, (tokens, heads, dim, _launch.elem(dtype)), _cache_args(k_cache, v_cache, k_scales, v_scales, heads, dim, CODES, d),
            _token_strides("k", k, k.shape, dtype, d), _token_strides("v", v, k.shape, dtype, d))


def paged_store_e4m3(k, v, k_cache, v_cache, k_scales, v_scales, slots, stream=None) -> None:
    """Quantise token i's keys and values (k, v: (tokens, kv_heads,
    head_dim), contiguous in the last dimension) into slot ``slots[i]`` (int32)
    of caches of codes; slots outside the caches (-1: padding) are skipped.  A
    block of positions whose first slot is written begins anew; the scale of
    one that is continued grows where the new tokens need it, and its codes
    with it.  Tokens of one block are neighbours in ``slots``, as
    PageTable.append gives them.  For serving: no gradient flows through the
    caches."""
    like = (_layout(k), _layout(v), _layout(k_cache), _layout(v_cache), _layout(k_scales), _layout(v_scales))
    known = _seen.get("store")
    if known is None or known[0] != like:
        known = like, _check_store(k, v, k_cache, v_cache, k_scales, v_scales)
        _seen["store"] = known
    d, sizes, cache, ks, vs = known[1]
    at = _launch.vector("slots", slots, sizes[0], torch.int32, d)
    cache = _with_addresses(cache, k_cache, v_cache, k_scales, v_scales)
    _launch.call(lib().spmv_paged_store_e4m3, "spmv_paged_store_e4m3", d, *sizes, at, ctypes.byref(cache), k.data_ptr(), ks,
                 v.data_ptr(), vs, _launch.handle(stream, d))


def _check_load(k_cache, v_cache, table, token_ptr, tokens, k_scales, v_scales, dtype, k, v):
    if not k_cache.is_cuda:
        raise TypeError("k_cache must be a CUDA tensor")
    d, codes = k_cache.device, k_cache.dtype == CODES
    if k_cache.dim() != 4:
        raise ValueError("k_cache must be (pages, page_size, kv_heads, head_dim)")
    if codes and dtype is None:
        raise TypeError("a cache of codes needs the dtype of the rows")
    if not codes and (k_scales is not None or v_scales is not None):
        raise TypeError(f"scales are of {CODES} caches, got {k_cache.dtype}")
    if not codes and dtype not in (None, k_cache.dtype):
        raise TypeError(f"a cache of {k_cache.dtype} is copied as it is, not to {dtype}")
    dtype = dtype or k_cache.dtype
    elem = _launch.elem(dtype)
    heads, dim = k_cache.shape[2:]
    if tokens < 0:
        raise ValueError("tokens must not be negative")
    shape = (tokens, heads, dim)
    cache = _cache_args(k_cache, v_cache, k_scales, v_scales, heads, dim, k_cache.dtype, d)
    if table.dim() != 2:
        raise ValueError("table must be (requests, max_pages)")
    requests = token_ptr.numel() - 1
    if requests < 0 or table.shape[0] < requests:
        raise ValueError("token_ptr must have an entry more than there are requests, and table a row for each")
    _launch.counts(requests, tokens, table.shape[1])
    stride = _launch.rows("table", table, table.shape, torch.int32, d)
    _launch.vector("token_ptr", token_ptr, requests + 1, torch.int32, d)
    dense = _I64x2(heads * dim, dim)
    ks, vs = (dense if t is None else _token_strides(name, t, shape, dtype, d) for name, t in (("k", k), ("v", v)))
    return d, dtype, shape, (requests, *shape, elem), (stride, table.shape[1]), cache, ks, vs


def paged_load(k_cache, v_cache, table, token_ptr, tokens: int, k_scales=None, v_scales=None, dtype=None, k=None, v=None, stream=None):
    """(k, v), (tokens, kv_heads, head_dim) each: rows ``token_ptr[r]`` ..
    ``token_ptr[r + 1] - 1`` (int32, requests + 1 entries) are positions 0, 1,
    ... of request r, whose pages are row r of ``table`` (int32).  Caches of
    codes need their scales and the rows' ``dtype``; others are copied.  Rows
    behind the last request, if ``tokens`` are more, are left as they were.  It
    has no derivative."""
    if _launch.tracked(k_cache, v_cache, k_scales, v_scales, k, v):
        _launch.no_outputs_given("paged_load", k, v)
        with _launch.on(stream, k_cache.device):
            return _launch.NoDerivative.apply(
                "paged_load", lambda: _load(k_cache, v_cache, table, token_ptr, tokens, k_scales, v_scales, dtype, None, None, None),
                k_cache, v_cache, k_scales, v_scales)
    return _load(k_cache, v_cache, table, token_ptr, tokens, k_scales, v_scales, dtype, k, v, stream)


def _load(k_cache, v_cache, table, token_ptr, tokens, k_scales, v_scales, dtype, k, v, stream):
    like = (_layout(k_cache), _layout(v_cache), _layout(table), _layout(token_ptr), tokens, _layout(k_scales), _layout(v_scales),
            dtype, _layout(k), _layout(v))
    known = _seen.get("load")
    if known is None or known[0] != like:
        known = like, _check_load(k_cache, v_cache, table, token_ptr, tokens, k_scales, v_scales, dtype, k, v)
        _seen["load"] = known
    d, dtype, shape, sizes, of_table, cache, ks, vs = known[1]
    if k is None:
        k = _launch.empty(stream, d, shape, dtype)
    if v is None:
        v = _launch.empty(stream, d, shape, dtype)
    cache = _with_addresses(cache, k_cache, v_cache, k_scales, v_scales)
    _launch.call(lib().spmv_paged_load, "spmv_paged_load", d, *sizes, table.data_ptr(), *of_table, token_ptr.data_ptr(),
                 ctypes.byref(cache), k.data_ptr(), ks, v.data_ptr(), vs, _launch.handle(stream, d))
    return k, v


class PagedAttentionE4M3(PagedAttention):
    """Attention of one new token for each of up to ``max_batch`` requests
    over caches of codes; ``dtype`` (bfloat16 or float16) is that of q and out.
    Keeps the workspace that joins requests cut between blocks: calls that may
    overlap on the GPU (two streams) need objects of their own, and an object
    is kept until its calls have run."""

    _workspace_of, _cache_dtype = "spmv_paged_attention_e4m3_workspace", CODES

    def __call__(self, q, k_cache, v_cache, k_scales, v_scales, table, lens, scale=None, out=None, lse=None, stream=None):
        """(out, lse) of q (batch, q_heads, head_dim) over the first
        ``lens[b]`` (int32) positions of each request, whose pages are row b
        of ``table`` (int32).  ``scale``: head_dim ** -0.5 if None.  It has no
        derivative."""
        scales = k_scales, v_scales
        if k_scales is None or v_scales is None:
            raise TypeError("k_scales and v_scales must be float32 tensors")
        if _launch.tracked(q, k_cache, v_cache, k_scales, v_scales, out):
            _launch.no_outputs_given("PagedAttentionE4M3", out, lse)
            with _launch.on(stream, self.device):
                return _launch.NoDerivative.apply(
                    "PagedAttentionE4M3", lambda: self._attend(q, k_cache, v_cache, table, lens, scale, scales=scales),
                    q, k_cache, v_cache, k_scales, v_scales)
        return self._attend(q, k_cache, v_cache, table, lens, scale, out, lse, stream, scales)

    def _check_scales(self, k_cache, scales):
        k_scales, v_scales = scales
        block = _scale_block(k_cache, k_scales, v_scales, self.device)
        self._scale_layout = block, _I64x3(*k_scales.stride()), _I64x3(*v_scales.stride())

    def _launch_with(self, scales, stream):
        block, ks, vs = self._scale_layout
        _launch.call(self._L.spmv_paged_attention_e4m3, "spmv_paged_attention_e4m3", self.device, self._args_ref, block,
                     scales[0].data_ptr(), ks, scales[1].data_ptr(), vs, _launch.handle(stream, self.device))
