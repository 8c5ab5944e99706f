"""Tokens sorted by expert and back, with the router's weights, and the gradient.

    route = lb.ExpertRoute(max_tokens, top_k, experts)   # keeps the index arrays and the workspace
    route.build(expert_ids)                              # (tokens, top_k) int32 or int64
    xs = route.dispatch(x)                               # (tokens * top_k, hidden), expert by expert
    ...                                                  # the experts' products over expert_ptr
    y = route.combine(ys, weights)                       # (tokens, hidden)
    dys, dw = route.combine_backward(dy, ys, weights)
    dx = route.dispatch_backward(dxs)

Argument marshalling only; include/spmv.h (spmv_route_*) has the contract.
"""
from __future__ import annotations

import ctypes

import torch

from . import _launch

__all__ = ["ExpertRoute"]


class ExpertRoute:
    """The routing of up to ``max_tokens`` tokens to ``top_k`` of ``experts``
    experts each.  ``build`` fills ``expert_ptr`` (experts + 1), ``entry``
    (tokens * top_k) and ``slot`` (tokens, top_k), int32; the other methods
    read ``slot``.  A route is rebuilt for each batch; it must not be rebuilt
    on one stream while another still uses it, and a training step keeps one
    per layer until its backward pass."""

    def __init__(self, max_tokens: int, top_k: int, experts: int, device="cuda"):
        from . import check, lib
        self._L = L = lib()
        size = ctypes.c_size_t()
        check(L.spmv_route_workspace(max_tokens, top_k, experts, ctypes.byref(size)), "spmv_route_workspace")
        self.device = _launch.cuda_device(device)
        self.max_tokens, self.top_k, self.experts = int(max_tokens), int(top_k), int(experts)
        n = self.max_tokens * self.top_k
        int32 = dict(dtype=torch.int32, device=self.device)
        self.expert_ptr = torch.empty(self.experts + 1, **int32)
        self._entry, self._slot = torch.empty(n, **int32), torch.empty(n, **int32)
        # fewer tokens never need more workspace
        self._workspace = torch.empty(size.value, dtype=torch.uint8, device=self.device)
        self._pointers = (self.expert_ptr.data_ptr(), self._entry.data_ptr() or None, self._slot.data_ptr() or None,
                          self._workspace.data_ptr() or None, size.value)
        self.tokens = None
        self.entry = self.slot = None

    def build(self, expert_ids, stream=None) -> "ExpertRoute":
        """Sort the entries of ``expert_ids`` (tokens, top_k) by expert; ids
        outside [0, experts) are dropped."""
        ids = expert_ids
        if ids.dtype not in (torch.int32, torch.int64) or ids.device != self.device:
            raise TypeError(f"expert_ids must be an int32 or int64 tensor on {self.device}")
        if ids.dim() != 2 or ids.shape[1] != self.top_k or ids.shape[0] > self.max_tokens:
            raise ValueError(f"expert_ids must be (tokens <= {self.max_tokens}, {self.top_k}), got {tuple(ids.shape)}")
        tokens, k = ids.shape
        ld = _launch.rows("expert_ids", ids, ids.shape, ids.dtype, self.device)
        ptr, entry, slot, work, size = self._pointers
        _launch.call(self._L.spmv_route_build, "spmv_route_build", self.device, tokens, k, self.experts,
                     ids.data_ptr() or None, ids.element_size(), ld, ptr, entry, slot, work, size,
                     _launch.handle(stream, self.device))
        if tokens != self.tokens:
            self.entry, self.slot = self._entry[:tokens * k], self._slot[:tokens * k].view(tokens, k)
            self.tokens = tokens
        return self

    def _built(self) -> int:
        if self.tokens is None:
            raise RuntimeError("the route has not been built")
        return self.tokens

    def _weights(self, weights):
        if weights is None:
            return None, 0
        ld = _launch.rows("weights", weights, (self.tokens, self.top_k), torch.float32, self.device)
        return weights.data_ptr() or None, ld

    def dispatch(self, x, out=None, stream=None):
        """xs[p] = x[entry[p] // top_k]; rows of dropped entries are zero."""
        t, k, d = self._built(), self.top_k, self.device
        e, hidden = _launch.elem(x.dtype), x.shape[-1]
        ldx = _launch.rows("x", x, (t, hidden), x.dtype, d)
        if out is None:
            out = _launch.empty(stream, d, (t * k, hidden), x.dtype)
        ldo = _launch.rows("out", out, (t * k, hidden), x.dtype, d)
        _launch.call(self._L.spmv_route_dispatch, "spmv_route_dispatch", d, t, k, hidden, e, self._pointers[2],
                     x.data_ptr() or None, ldx, out.data_ptr() or None, ldo, _launch.handle(stream, d))
        return out

    def combine(self, ys, weights=None, out=None, stream=None):
        """y[t] = sum over j of weights[t, j] * ys[slot[t, j]] (weights float32; None: 1)."""
        t, k, d = self._built(), self.top_k, self.device
        e, hidden = _launch.elem(ys.dtype), ys.shape[-1]
        ldys = _launch.rows("ys", ys, (t * k, hidden), ys.dtype, d)
        w, ldw = self._weights(weights)
        if out is None:
            out = _launch.empty(stream, d, (t, hidden), ys.dtype)
        ldo = _launch.rows("out", out, (t, hidden), ys.dtype, d)
        _launch.call(self._L.spmv_route_combine, "spmv_route_combine", d, t, k, hidden, e, self._pointers[2], w, ldw,
                     ys.data_ptr() or None, ldys, out.data_ptr() or None, ldo, _launch.handle(stream, d))
        return out

    def dispatch_backward(self, dxs, out=None, stream=None):
        """The gradient of dispatch: dx[t] = sum over j of dxs[slot[t, j]]."""
        return self.combine(dxs, None, out, stream)

    def combine_backward(self, dy, ys, weights=None, out=None, dweights=None, stream=None):
        """The gradient of combine: (dys, dweights).  ``out`` may be ``ys``."""
        t, k, d = self._built(), self.top_k, self.device
        e, hidden = _launch.elem(dy.dtype), dy.shape[-1]
        lddy = _launch.rows("dy", dy, (t, hidden), dy.dtype, d)
        ldys = _launch.rows("ys", ys, (t * k, hidden), dy.dtype, d)
        w, ldw = self._weights(weights)
        if out is None:
            out = _launch.empty(stream, d, (t * k, hidden), dy.dtype)
        if dweights is None:
            dweights = _launch.empty(stream, d, (t, k), torch.float32)
        ldo = _launch.rows("out", out, (t * k, hidden), dy.dtype, d)
        lddw = _launch.rows("dweights", dweights, (t, k), torch.float32, d)
        _launch.call(self._L.spmv_route_combine_backward, "spmv_route_combine_backward", d, t, k, hidden, e,
                     self._pointers[2], w, ldw, dy.data_ptr() or None, lddy, ys.data_ptr() or None, ldys,
                     out.data_ptr() or None, ldo, dweights.data_ptr() or None, lddw, _launch.handle(stream, d))
        return out, dweights
