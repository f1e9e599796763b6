"""Argument checks shared by the layers' Python entry points.

The C entry points check sizes, alignment and scalars, but a pointer says nothing
about a tensor's device, type or shape: that is checked here, before the call.  A
serving step is a few microseconds of GPU work, so a tensor that is as it should be
costs one short expression, and only a wrong one pays for its message.
"""

from __future__ import annotations

import functools
import inspect

import torch

from . import dr

DTYPES = {torch.float32: dr.DR_FP32, torch.bfloat16: dr.DR_BF16}

_current_device = torch._C._cuda_getDevice
_current_stream = torch._C._cuda_getCurrentRawStream


def _refuse(t, name, shape, dtype, device, contiguous):
    if not torch.is_tensor(t):
        raise TypeError(f"{name} must be a tensor, got {type(t).__name__}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda or t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{device}")
    if contiguous:
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} must have contiguous channels (last stride 1)")


def check(t, name, shape, dtype, device):
    """``t`` must be a contiguous tensor of this shape and type on CUDA device ``device``."""
    try:
        if (t.shape == shape and t.dtype is dtype and t.is_cuda and t.get_device() == device
                and t.is_contiguous()):
            return
    except AttributeError:
        pass
    _refuse(t, name, shape, dtype, device, True)


def check_rows(t, name, shape, dtype, device):
    """As ``check``, but only the last dimension has to be contiguous."""
    try:
        if (t.shape == shape and t.dtype is dtype and t.is_cuda and t.get_device() == device
                and (t.stride(-1) == 1 or t.shape[-1] == 1)):
            return
    except AttributeError:
        pass
    _refuse(t, name, shape, dtype, device, False)


def activations(t, name, dims):
    """(dr_dtype, CUDA device) of a tensor with ``dims`` dimensions and contiguous channels."""
    if not torch.is_tensor(t):
        raise TypeError(f"{name} must be a tensor, got {type(t).__name__}")
    code = DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got {t.dim()}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name} must have contiguous channels (last stride 1)")
    return code, t.get_device()


def ptr(t):
    return None if t is None else t.data_ptr()


def call(name, device, fn, *args):
    """``fn(*args, stream)`` with ``device`` current, on its current stream; raises
    ``dr.DrError`` for a status other than DR_OK."""
    if device != _current_device():
        with torch.cuda.device(device):
            return call(name, device, fn, *args)
    status = fn(*args, _current_stream(device))
    if status:
        dr.check(status, name)


def on_stream(fn):
    """With a ``stream``, of the device of ``fn``'s first tensor (a torch stream or a raw handle),
    ``fn`` runs as if that were the current one: what it allocates belongs to that stream, so
    neither its scratch nor its outputs are memory that the current stream still uses or may be
    given while the call's kernels run.  The memory of tensors that are passed in is not given
    to others either before what the call put on the stream is done; that they are ready when
    the stream gets there is the caller's part."""
    first = next(iter(inspect.signature(fn).parameters))

    @functools.wraps(fn)
    def run(*args, **kw):
        stream = kw.get("stream")
        if stream is None:
            return fn(*args, **kw)
        kw["stream"] = None
        device = getattr(args[0] if args else kw.get(first), "device", None)
        if device is None or device.type != "cuda":
            return fn(*args, **kw)   # refused there
        if not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(stream, device=device)
        elif stream.device != device:
            raise ValueError(f"stream is on {stream.device}, the tensors are on {device}")
        with torch.cuda.stream(stream):
            result = fn(*args, **kw)
        for t in (*args, *kw.values(), *(kw.get("grads") or {}).values()):
            if torch.is_tensor(t):
                t.record_stream(stream)
        return result
    return run


def scratch(size_of, description, x, device, workspace):
    """(tensor or None, bytes) of a call's workspace.  "auto" allocates what ``size_of`` asks
    for, None goes without one, or a contiguous uint8 tensor on x's device to reuse."""
    if workspace is None:
        return None, 0
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError('workspace must be "auto", None or a uint8 tensor')
        if device != _current_device():
            with torch.cuda.device(device):
                n = size_of(description)
        else:
            n = size_of(description)
        return (torch.empty(n, dtype=torch.uint8, device=x.device), n) if n else (None, 0)
    check(workspace, "workspace", (workspace.numel(),), torch.uint8, device)
    return workspace, workspace.numel()
