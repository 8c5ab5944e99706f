"""Attention of packed prompts.

    attend = lb.PromptAttention(max_requests, q_heads, kv_heads, head_dim, torch.bfloat16)
    out, lse = attend(q, k, v, pages.token_ptr)            # q: (tokens, q_heads, head_dim), k, v: (tokens, kv_heads, head_dim)
    out, lse = attend(q, k, v, pages.token_ptr, kv_ptr)    # chunks behind what their requests hold already

The second form takes every request's keys and values from its first position
on, as ``paged_load`` reads them back.  Argument marshalling only;
include/spmv.h (spmv_prompt_attention) has the contract.
"""
from __future__ import annotations

import ctypes

import torch

from . import _launch, lib
from .paged import _I64x2

__all__ = ["PromptAttention"]


class PromptAttentionArgs(ctypes.Structure):
    _fields_ = [("requests", ctypes.c_int32), ("tokens", ctypes.c_int32), ("keys", ctypes.c_int32),
                ("q_heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("elem", ctypes.c_int32), ("causal", ctypes.c_int32), ("scale", ctypes.c_float), ("reserved", ctypes.c_int32),
                ("q_stride", _I64x2), ("k_stride", _I64x2), ("v_stride", _I64x2), ("out_stride", _I64x2),
                ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("q_ptr", ctypes.c_void_p),
                ("kv_ptr", ctypes.c_void_p), ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p), ("status", ctypes.c_void_p),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t)]


class PromptAttention:
    """Attention of up to ``max_requests`` packed prompts, bfloat16 or
    float16.  Keeps the workspace that joins the shares of queries whose keys
    are cut between blocks: calls that may overlap on the GPU (two streams)
    need objects of their own, and an object is kept until its calls have
    run."""

    def __init__(self, max_requests: int, q_heads: int, kv_heads: int, head_dim: int, dtype, device="cuda"):
        self._L, self.device, self.dtype = lib(), _launch.cuda_device(device), dtype
        self._args = a = PromptAttentionArgs()
        a.elem = _launch.elem(dtype)
        if dtype == torch.float32:
            raise TypeError("prompts are attended to in bfloat16 or float16")
        self.max_requests = int(max_requests)
        self.q_heads, self.kv_heads, self.head_dim = int(q_heads), int(kv_heads), int(head_dim)
        _launch.counts(self.q_heads, self.kv_heads, self.head_dim)
        a.q_heads, a.kv_heads, a.head_dim = self.q_heads, self.kv_heads, self.head_dim
        size = ctypes.c_size_t()
        _launch.call(self._L.spmv_prompt_attention_workspace, "spmv_prompt_attention_workspace", self.device, self.q_heads,
                     self.kv_heads, self.head_dim, a.elem, ctypes.byref(size))
        self._workspace = torch.empty(size.value, dtype=torch.uint8, device=self.device)
        self._status = torch.zeros(1, dtype=torch.int32, device=self.device)
        a.status, a.workspace, a.workspace_bytes = self._status.data_ptr(), self._workspace.data_ptr(), size.value
        self._like = self._shape = None
        self._dense, self._scale, self._args_ref = False, self.head_dim ** -0.5, ctypes.byref(a)
        _launch.settle(self.device)

    def __call__(self, q, k, v, q_ptr, kv_ptr=None, causal=True, scale=None, out=None, lse=None, stream=None):
        """(out, lse) of queries q (tokens, q_heads, head_dim) over keys k and
        values v (keys, kv_heads, head_dim).  Request r's queries are rows
        ``q_ptr[r]`` .. ``q_ptr[r + 1] - 1`` (int32), its keys those of
        ``kv_ptr`` (None: the same rows).  Its last query stands at its last
        key; with ``causal`` a query sees the keys up to its own place.
        Rows and heads of q, k and v are multiples of 16 bytes apart, and not
        0 (expanded).
        ``scale``: head_dim ** -0.5 if None.  Rows of no request are left as
        they were.  It has no derivative."""
        if _launch.tracked(q, k, v, out):
            _launch.no_outputs_given("PromptAttention", out, lse)
            with _launch.on(stream, self.device):
                return _launch.NoDerivative.apply("PromptAttention", lambda: self._attend(q, k, v, q_ptr, kv_ptr, causal, scale), q, k, v)
        return self._attend(q, k, v, q_ptr, kv_ptr, causal, scale, out, lse, stream)

    def _attend(self, q, k, v, q_ptr, kv_ptr=None, causal=True, scale=None, out=None, lse=None, stream=None):
        d, a = self.device, self._args
        like = (q.shape, q.stride(), q.dtype, q.device, k.shape, k.stride(), k.dtype, k.device, v.shape, v.stride(), v.dtype, v.device,
                q_ptr.shape, q_ptr.stride(), q_ptr.dtype, q_ptr.device)
        if kv_ptr is not None:
            like += (kv_ptr.shape, kv_ptr.stride(), kv_ptr.dtype, kv_ptr.device)
        if like != self._like:
            self._like = None
            self._check(q, k, v, q_ptr, kv_ptr)
            self._like, self._shape, self._dense = like, (q.shape, q.shape[:2]), False
        shape, heads = self._shape
        if out is not None:
            if out.dtype != self.dtype or out.device != d or out.shape != shape or (out.stride(2) != 1 and out.numel()):
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
        a.causal = bool(causal)
        a.q, a.k, a.v, a.q_ptr = q.data_ptr(), k.data_ptr(), v.data_ptr(), q_ptr.data_ptr()
        a.kv_ptr = None if kv_ptr is None else kv_ptr.data_ptr()
        a.out, a.lse = out.data_ptr(), lse.data_ptr()
        _launch.call(self._L.spmv_prompt_attention, "spmv_prompt_attention", d, self._args_ref, _launch.handle(stream, d))
        return out, lse

    def _check(self, q, k, v, q_ptr, kv_ptr):
        """Checks the inputs' layouts and puts them into the arguments."""
        d, dtype, a = self.device, self.dtype, self._args
        for name, t, heads in (("q", q, self.q_heads), ("k", k, self.kv_heads), ("v", v, self.kv_heads)):
            if t.dtype != dtype or t.device != d:
                raise TypeError(f"{name} must be a {dtype} tensor on {d}, got {t.dtype} on {t.device}")
            if t.dim() != 3 or t.shape[1:] != (heads, self.head_dim):
                raise ValueError(f"{name} must be (tokens, {heads}, {self.head_dim}), got {tuple(t.shape)}")
            if t.stride(2) != 1 and t.numel():
                raise ValueError(f"{name} must have a contiguous last dimension")
        if k.shape != v.shape:
            raise ValueError("k and v differ in shape")
        if q_ptr.dim() != 1 or not 1 <= q_ptr.numel() <= self.max_requests + 1:
            raise ValueError(f"q_ptr must have an entry more than there are requests (at most {self.max_requests})")
        n = q_ptr.numel()
        _launch.vector("q_ptr", q_ptr, n, torch.int32, d)
        if kv_ptr is not None:
            _launch.vector("kv_ptr", kv_ptr, n, torch.int32, d)
        _launch.counts(n - 1, q.shape[0], k.shape[0])
        a.requests, a.tokens, a.keys = n - 1, q.shape[0], k.shape[0]
        a.q_stride[:], a.k_stride[:], a.v_stride[:] = q.stride()[:2], k.stride()[:2], v.stride()[:2]

    def device_status(self) -> int:
        """Flags of the calls so far (0 = none); waits for the device.  Bit 0:
        a request's queries, bit 1: its keys are not rows of the tensors; bit
        2: a wait inside the kernel ran out, and an output is not complete."""
        torch.cuda.synchronize(self.device)
        return int(self._status.item())
