"""Argument checks shared by the layers' Python entry points.

The C entry points check sizes, alignment and scalars, but a pointer says nothing
about a tensor's device, type or shape: that is checked here, before the call.
"""

from __future__ import annotations

import torch

from . import dr

DTYPES = {torch.float32: dr.DR_FP32, torch.bfloat16: dr.DR_BF16}


def check(t, name, shape, dtype, like, contiguous=True):
    """``t`` (None passes) must be a tensor of this shape and type on ``like``'s device."""
    if t is None:
        return
    if not torch.is_tensor(t):
        raise TypeError(f"{name} must be a tensor, got {type(t).__name__}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != like.device:
        raise ValueError(f"{name} is on {t.device}, expected {like.device}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def activations(t, name, dims):
    """The dr_dtype of a CUDA tensor with ``dims`` dimensions and contiguous channels."""
    if not torch.is_tensor(t):
        raise TypeError(f"{name} must be a tensor, got {type(t).__name__}")
    if t.dtype not in DTYPES:
        raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got {t.dim()}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must have contiguous channels (last stride 1)")
    return DTYPES[t.dtype]


def like_x(t, name, shape, x):
    """``t`` (None passes): x's type and device, this shape, contiguous channels."""
    if t is None:
        return
    check(t, name, shape, x.dtype, x, contiguous=False)
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must have contiguous channels (last stride 1)")


class launch:
    """The context of one call: its device is current, its stream as in ``dr``."""

    def __init__(self, x, stream):
        self.device, self.stream = torch.cuda.device(x.device), stream

    def __enter__(self):
        self.device.__enter__()
        return torch.cuda.current_stream().cuda_stream if self.stream is None else self.stream

    def __exit__(self, *exc):
        return self.device.__exit__(*exc)


def scratch(n_bytes, x, workspace):
    """The workspace of a call: "auto" allocates what the call asks for, None goes without
    one, or a contiguous uint8 tensor on x's device to reuse."""
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError('workspace must be "auto", None or a uint8 tensor')
        return torch.empty(n_bytes, dtype=torch.uint8, device=x.device) if n_bytes else None
    if workspace is not None:
        check(workspace, "workspace", workspace.shape, torch.uint8, x)
    return workspace


def size_of(workspace):
    return 0 if workspace is None else workspace.numel()
