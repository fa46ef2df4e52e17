"""Torch tensors as the C ABI takes them: pointers, dtype codes, the current
stream and workspaces, with the checks that only torch can make."""
from __future__ import annotations

import contextlib
from typing import Optional

import torch

from . import _abi


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("plp runs on the GPU only: got a CPU tensor")
    if not t.is_contiguous():
        raise ValueError("plp needs contiguous tensors")
    return t.data_ptr()


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return _abi.DTYPE_F32
    if t.dtype == torch.bfloat16:
        return _abi.DTYPE_BF16
    raise ValueError(f"unsupported dtype {t.dtype}: float32 or bfloat16")


def _stream(device: torch.device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _workspace(nbytes: int, device, workspace: Optional[torch.Tensor]) -> torch.Tensor:
    if workspace is not None:
        if workspace.numel() * workspace.element_size() < nbytes:
            raise ValueError(f"workspace too small: need {nbytes} bytes")
        return workspace
    return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)


def _check_vec(t, n, dtype, name):
    if t is None:
        return None
    if t.numel() != n or t.dtype != dtype:
        raise ValueError(f"{name}: expected {n} elements of {dtype}, got {tuple(t.shape)} {t.dtype}")
    return t


def _one_device(tensors) -> torch.device:
    """The GPU that all of (name, tensor or None) pairs are on."""
    dev, index = None, -1
    for name, t in tensors:
        if t is None:
            continue
        i = t.get_device()
        if i < 0:
            raise ValueError("plp runs on the GPU only: got a CPU tensor")
        if dev is None:
            dev, index = t.device, i
        elif i != index:
            raise ValueError(f"{name} is on {t.device}, the other tensors on {dev}")
    return dev


# The current stream's handle without a Stream object around it: a tenth of a
# microsecond instead of two.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_on(device: torch.device) -> int:
    return _raw_stream(device.index) if _raw_stream is not None else _stream(device)


_STAY = contextlib.nullcontext()


def _on(device: torch.device):
    """The device as the current one, for the launches of a call."""
    return _STAY if torch.cuda.current_device() == device.index else torch.cuda.device(device)
