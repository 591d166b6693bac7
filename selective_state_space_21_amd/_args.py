"""Checks and marshalling of tensor arguments, shared by the package's
wrappers: types, shapes and dtypes first, then devices and layout, before
anything reaches the library.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import _native

DTYPES = {torch.float32: _native.SSM_F32, torch.bfloat16: _native.SSM_BF16}


def ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _dev_tensor(name, t, dtype=None, device=None):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a device tensor (got {t.device})")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def check_args(device, *specs) -> None:
    """specs: (name, tensor or None, expected shape, dtype).  Types, shapes and
    dtypes of every argument are checked first, then device and contiguity."""
    for _name, t, shape, dtype in specs:      # all as they should be: one pass
        if t is not None and not (
                isinstance(t, torch.Tensor) and t.shape == shape and (dtype is None or t.dtype is dtype)
                and t.is_cuda and (device is None or t.device == device) and t.is_contiguous()):
            break
    else:
        return
    for name, t, shape, dtype in specs:
        if t is None:
            continue
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
        if dtype is not None and t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    for name, t, _shape, dtype in specs:
        _dev_tensor(name, t, dtype, device)


def check_workspace(ws, need: int, device):
    """A caller-supplied workspace: a contiguous uint8 tensor on the call's
    device holding at least `need` bytes, or None."""
    if ws is None:
        return None
    if not isinstance(ws, torch.Tensor):
        raise TypeError("workspace must be a torch.Tensor")
    if ws.dtype != torch.uint8:
        raise TypeError(f"workspace must be uint8 (got {ws.dtype})")
    if ws.numel() < need:
        raise ValueError(f"workspace holds {ws.numel()} bytes, the call needs {need}")
    if ws.device.type != "cuda" or ws.device != device:
        raise ValueError(f"workspace is on {ws.device}, expected {device}")
    if not ws.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return ws


def workspace(ws, need: int, device):
    ws = check_workspace(ws, need, device)
    if need and ws is None:
        ws = torch.empty(need, dtype=torch.uint8, device=device)
    return ws, (0 if ws is None else ws.numel())


def act_dtype(name, t):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in DTYPES:
        raise TypeError(f"{name} must be float32 or bfloat16 (got {t.dtype})")
    return t.dtype


def stream_handle(device) -> int:
    """The hipStream_t of torch's current stream on the device (the raw handle
    where torch gives it, which costs a tenth of making a Stream object)."""
    if _raw_stream is not None and device.index is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def need(**given) -> None:
    """Raises for a required tensor that is missing."""
    for name, t in given.items():
        if t is None:
            raise TypeError(f"{name} must be a torch.Tensor")
