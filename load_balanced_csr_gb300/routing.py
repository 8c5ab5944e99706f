"""Tokens sorted by expert and back, with the router's weights, and the gradient.

    route = lb.ExpertRoute(max_tokens, top_k, experts)   # keeps the index arrays and the workspace
    route.build(expert_ids)                              # (tokens, top_k) int32 or int64
    xs = route.dispatch(x)                               # (tokens * top_k, hidden), expert by expert
    ...                                                  # the experts' products over expert_ptr
    y = route.combine(ys, weights)                       # (tokens, hidden)
    dys, dw = route.combine_backward(dy, ys, weights)
    dx = route.dispatch_backward(dxs)

dispatch and combine are differentiable: torch's backward pass calls the two
gradients above, on the stream of the forward call.  The forward call keeps a
copy of ``slot`` for it, so the route may be rebuilt in between.  Argument
marshalling only; include/spmv.h (spmv_route_*) has the contract.
"""
from __future__ import annotations

import ctypes

import torch
from torch.autograd.function import once_differentiable

from . import _launch

__all__ = ["ExpertRoute"]


def _contiguous_rows(g):
    # torch's gradients may be expanded or transposed
    return g if g.stride(-1) == 1 or g.shape[-1] == 1 else g.contiguous()


def _at(slot):
    return slot.shape[0], slot.data_ptr()


class _Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, route, slot):
        ctx.route = route
        ctx.save_for_backward(slot)
        return route._dispatch(_at(slot), x)

    @staticmethod
    def backward(ctx, dxs):
        return _Sum.apply(_contiguous_rows(dxs), ctx.route, *ctx.saved_tensors), None, None


class _Sum(torch.autograd.Function):
    """combine without weights: dispatch's gradient, and its gradient is dispatch."""

    @staticmethod
    def forward(ctx, ys, route, slot):
        ctx.route = route
        ctx.save_for_backward(slot)
        return route._combine(_at(slot), ys)

    @staticmethod
    def backward(ctx, dy):
        return _Dispatch.apply(_contiguous_rows(dy), ctx.route, *ctx.saved_tensors), None, None


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ys, weights, route, slot):
        ctx.route = route
        ctx.save_for_backward(ys, weights, slot)
        return route._combine(_at(slot), ys, weights)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        ys, weights, slot = ctx.saved_tensors
        return *ctx.route._combine_backward(_at(slot), _contiguous_rows(dy), ys, weights), None, None


class ExpertRoute:
    """The routing of up to ``max_tokens`` tokens to ``top_k`` of ``experts``
    experts each.  ``build`` fills ``expert_ptr`` (experts + 1), ``entry``
    (tokens * top_k) and ``slot`` (tokens, top_k), int32; the other methods
    read ``slot``.  A route is rebuilt for each batch; it must not be rebuilt
    on one stream while another still uses it, and a training step that calls
    the gradients itself keeps one per layer until its backward pass.  Keep it
    until its calls have run."""

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
        # fewer tokens never need more workspace (spmv_route_workspace)
        self._workspace = torch.empty(size.value, dtype=torch.uint8, device=self.device)
        self._pointers = (self.expert_ptr.data_ptr(), self._entry.data_ptr(), self._slot.data_ptr(),
                          self._workspace.data_ptr(), size.value)
        self.tokens = None
        self.entry = self.slot = None
        # the layouts of each method's tensors that were checked last, and what the checks gave
        self._seen = {}
        _launch.settle(self.device)

    def build(self, expert_ids, stream=None) -> "ExpertRoute":
        """Sort the entries of ``expert_ids`` (tokens, top_k) by expert; ids
        outside [0, experts) are dropped."""
        ids, d = expert_ids, self.device
        like = (ids.shape, ids.stride(), ids.dtype, ids.device)
        known = self._seen.get("build")
        if known is None or known[0] != like:
            if ids.dtype not in (torch.int32, torch.int64) or ids.device != d:
                raise TypeError(f"expert_ids must be an int32 or int64 tensor on {d}")
            if ids.dim() != 2 or ids.shape[1] != self.top_k or ids.shape[0] > self.max_tokens:
                raise ValueError(f"expert_ids must be (tokens <= {self.max_tokens}, {self.top_k}), got {tuple(ids.shape)}")
            known = like, ids.shape[0], ids.element_size(), _launch.rows("expert_ids", ids, ids.shape, ids.dtype, d)
            self._seen["build"] = known
        _, tokens, size, ld = known
        ptr, entry, slot, work, room = self._pointers
        _launch.call(self._L.spmv_route_build, "spmv_route_build", d, tokens, self.top_k, self.experts,
                     ids.data_ptr(), size, ld, ptr, entry, slot, work, room, _launch.handle(stream, d))
        if tokens != self.tokens:
            n = tokens * self.top_k
            self.entry, self.slot = self._entry[:n], self._slot[:n].view(tokens, self.top_k)
            self.tokens = tokens
        return self

    def _built(self):
        """The tokens and where their slots are."""
        if self.tokens is None:
            raise RuntimeError("the route has not been built")
        return self.tokens, self._pointers[2]

    def _kept_slot(self):
        self._built()
        return self.slot.clone()

    def _rows(self, what, like, *given):
        """The element type, hidden size and row strides of a call's tensors
        (name, tensor or None, rows), the first of which sets the type and
        the hidden size; `like` is what they depend on."""
        (_, first, _), found = given[0], []
        hidden = first.shape[-1] if first.dim() else 0
        for name, x, rows in given:
            found.append(hidden if x is None else _launch.rows(name, x, (rows, hidden), first.dtype, self.device))
        known = self._seen[what] = (like, _launch.elem(first.dtype), hidden, *found)
        return known

    def _weights(self, tokens, weights):
        if weights is None:
            return 0, 0
        like = (tokens, weights.shape, weights.stride(), weights.dtype, weights.device)
        known = self._seen.get("weights")
        if known is None or known[0] != like:
            ld = _launch.rows("weights", weights, (tokens, self.top_k), torch.float32, self.device)
            known = self._seen["weights"] = (like, ld)
        return weights.data_ptr(), known[1]

    def dispatch(self, x, out=None, stream=None):
        """xs[p] = x[entry[p] // top_k]; rows of dropped entries are zero."""
        if _launch.tracked(x, out):
            _launch.no_outputs_given("dispatch", out)
            with _launch.on(stream, self.device):
                return _Dispatch.apply(x, self, self._kept_slot())
        return self._dispatch(self._built(), x, out, stream)

    def _dispatch(self, at, x, out=None, stream=None):
        (t, slot), k, d = at, self.top_k, self.device
        like = (t, x.shape, x.stride(), x.dtype, x.device,
                None if out is None else (out.shape, out.stride(), out.dtype, out.device))
        known = self._seen.get("dispatch")
        if known is None or known[0] != like:
            known = self._rows("dispatch", like, ("x", x, t), ("out", out, t * k))
        _, e, hidden, ldx, ldo = known
        if out is None:
            out = _launch.empty(stream, d, (t * k, hidden), x.dtype)
        _launch.call(self._L.spmv_route_dispatch, "spmv_route_dispatch", d, t, k, hidden, e, slot,
                     x.data_ptr(), ldx, out.data_ptr(), ldo, _launch.handle(stream, d))
        return out

    def combine(self, ys, weights=None, out=None, stream=None):
        """y[t] = sum over j of weights[t, j] * ys[slot[t, j]] (weights float32; None: 1)."""
        if _launch.tracked(ys, weights, out):
            _launch.no_outputs_given("combine", out)
            with _launch.on(stream, self.device):
                slot = self._kept_slot()
                return _Sum.apply(ys, self, slot) if weights is None else _Combine.apply(ys, weights, self, slot)
        return self._combine(self._built(), ys, weights, out, stream)

    def _combine(self, at, ys, weights=None, out=None, stream=None):
        (t, slot), k, d = at, self.top_k, self.device
        like = (t, ys.shape, ys.stride(), ys.dtype, ys.device,
                None if out is None else (out.shape, out.stride(), out.dtype, out.device))
        known = self._seen.get("combine")
        if known is None or known[0] != like:
            known = self._rows("combine", like, ("ys", ys, t * k), ("out", out, t))
        _, e, hidden, ldys, ldo = known
        w, ldw = self._weights(t, weights)
        if out is None:
            out = _launch.empty(stream, d, (t, hidden), ys.dtype)
        _launch.call(self._L.spmv_route_combine, "spmv_route_combine", d, t, k, hidden, e, slot, w, ldw,
                     ys.data_ptr(), ldys, out.data_ptr(), ldo, _launch.handle(stream, d))
        return out

    def dispatch_backward(self, dxs, out=None, stream=None):
        """The gradient of dispatch: dx[t] = sum over j of dxs[slot[t, j]]."""
        return self.combine(dxs, None, out, stream)

    def combine_backward(self, dy, ys, weights=None, out=None, dweights=None, stream=None):
        """The gradient of combine: (dys, dweights).  ``out`` may be ``ys``.
        It has no derivative of its own."""
        if _launch.tracked(dy, ys, weights, out, dweights):
            _launch.no_outputs_given("combine_backward", out, dweights)
            with _launch.on(stream, self.device):
                return _launch.NoDerivative.apply(
                    "combine_backward", lambda: self._combine_backward(self._built(), dy, ys, weights), dy, ys, weights)
        return self._combine_backward(self._built(), dy, ys, weights, out, dweights, stream)

    def _combine_backward(self, at, dy, ys, weights=None, out=None, dweights=None, stream=None):
        (t, slot), k, d = at, self.top_k, self.device
        like = (t, dy.shape, dy.stride(), dy.dtype, dy.device, ys.shape, ys.stride(), ys.dtype, ys.device,
                None if out is None else (out.shape, out.stride(), out.dtype, out.device))
        known = self._seen.get("combine_backward")
        if known is None or known[0] != like:
            known = self._rows("combine_backward", like, ("dy", dy, t), ("ys", ys, t * k), ("out", out, t * k))
        _, e, hidden, lddy, ldys, ldo = known
        w, ldw = self._weights(t, weights)
        if out is None:
            out = _launch.empty(stream, d, (t * k, hidden), dy.dtype)
        if dweights is None:
            dweights, lddw = _launch.empty(stream, d, (t, k), torch.float32), k
        else:
            lddw = _launch.rows("dweights", dweights, (t, k), torch.float32, d)
        _launch.call(self._L.spmv_route_combine_backward, "spmv_route_combine_backward", d, t, k, hidden, e,
                     slot, w, ldw, dy.data_ptr(), lddy, ys.data_ptr(), ldys, out.data_ptr(), ldo,
                     dweights.data_ptr(), lddw, _launch.handle(stream, d))
        return out, dweights
