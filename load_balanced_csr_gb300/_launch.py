"""Shared by the language-model operators' bindings: streams, outputs, checks."""
from __future__ import annotations

import contextlib

import torch
import torch.autograd.forward_ad as _forward_mode

ELEMS = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}

_raw_stream = torch._C._cuda_getCurrentRawStream


def elem(dtype) -> int:
    try:
        return ELEMS[dtype]
    except KeyError:
        raise TypeError(f"elements must be float32, bfloat16 or float16, got {dtype}") from None


def handle(stream, device) -> int:
    """The cudaStream_t of ``stream`` (None: the device's current stream)."""
    if stream is None:
        return _raw_stream(device.index)
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def on(stream, device):
    """A context with ``stream`` current (None: as it is)."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(handle(stream, device), device=device)
    return torch.cuda.stream(stream)


def empty(stream, device, shape, dtype):
    """An output for a launch on ``stream``, taken from that stream's own
    memory: memory of another stream could still be in use there."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with on(stream, device):
        return torch.empty(shape, dtype=dtype, device=device)


def tracked(*tensors) -> bool:
    """Whether torch differentiates a call on these tensors (or None)."""
    if torch.is_grad_enabled():
        for t in tensors:
            if t is not None and t.requires_grad:
                return True
    if _forward_mode._current_level < 0:
        return False
    return any(t is not None and _forward_mode.unpack_dual(t).tangent is not None for t in tensors)


def no_outputs_given(what, *given) -> None:
    """Refuses outputs of the caller's for a call that torch differentiates, as torch's own operators do."""
    if any(t is not None for t in given):
        raise RuntimeError(f"{what}: outputs given by the caller (out=...) have no gradient, but a tensor of the call "
                           "requires one")


class NoDerivative(torch.autograd.Function):
    """run()'s outputs, which raise an error when a gradient through them is asked for."""

    @staticmethod
    def forward(ctx, what, run, *tensors):
        ctx.what = what
        return run()

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError(f"{ctx.what} has no derivative")


def settle(device) -> None:
    """Waits for the device's current stream: the last step of a constructor.
    What it set is then set for every stream, and no earlier user of the
    memory it took is still at work.  (While the stream is captured nothing
    has run and the object belongs to the graph.)"""
    stream = torch.cuda.current_stream(device)
    with torch.cuda.stream(stream):
        capturing = torch.cuda.is_current_stream_capturing()
    if not capturing:
        stream.synchronize()


_current_device = torch._C._cuda_getDevice


def call(fn, what, device, *args) -> None:
    """One library call with ``device`` current; raises SpmvError."""
    if device.index == _current_device():
        status = fn(*args)
    else:
        with torch.cuda.device(device):
            status = fn(*args)
    if status:
        from . import check
        check(status, what)


def cuda_device(device):
    """``device`` with its index filled in."""
    device = torch.device(device)
    if device.type != "cuda":
        raise TypeError("a CUDA device is needed")
    return device if device.index is not None else torch.device("cuda", torch.cuda.current_device())


def rows(name, t, shape, dtype, device):
    """Checks a row-major matrix (unit stride in a row) and returns its row stride."""
    if t.dtype != dtype or t.device != device:
        raise TypeError(f"{name} must be a {dtype} tensor on {device}, got {t.dtype} on {t.device}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    ld, unit = t.stride()
    if unit != 1 and shape[1] > 1 and shape[0] > 0:
        raise ValueError(f"{name} must have contiguous rows")
    return ld if shape[0] > 1 else max(ld, shape[1])


def vector(name, t, n, dtype, device):
    """Checks a contiguous vector of at least n entries."""
    if t.dtype != dtype or t.device != device:
        raise TypeError(f"{name} must be a {dtype} tensor on {device}, got {t.dtype} on {t.device}")
    if t.dim() != 1 or t.numel() < n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous vector of at least {n} entries")
    return t.data_ptr()
