"""Argument checks and marshalling shared by the binding's modules."""

from __future__ import annotations

import torch

_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


# The handle alone: building the torch.cuda.Stream object took 2 us a call.
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else None


def _stream(t: torch.Tensor) -> int:
    if _raw_stream is None:
        return torch.cuda.current_stream(t.device).cuda_stream
    return _raw_stream(t.get_device())


def _rows(x: torch.Tensor, name: str):
    """(n, v, ld) of a 2-D tensor whose rows are contiguous."""
    if x.dim() != 2:
        raise ValueError(f"{name} must be 2-D [N, V], got shape {tuple(x.shape)}")
    n, v = x.shape
    ld, step = x.stride()
    if v > 1 and step != 1:
        raise ValueError(f"{name} rows must be contiguous (stride(1) == 1)")
    if n <= 1:
        ld = max(v, ld)
    if ld < v:
        raise ValueError(f"{name} row stride {ld} is smaller than its width {v}")
    return n, v, ld


def _vec(t: torch.Tensor, name: str, n: int, dtype: torch.dtype) -> None:
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != (n,):
        raise ValueError(f"{name} must have shape [{n}], got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _cuda(*ts) -> None:
    for t in ts:
        if not t.is_cuda:
            raise ValueError("all tensors must be CUDA tensors")


def _workspace(t: torch.Tensor):
    """(pointer, bytes) of a scratch tensor.  A strided or expanded one would not own
    the bytes that its element count gives, and the kernels would write past it."""
    if not t.is_contiguous():
        raise ValueError("workspace must be contiguous")
    _cuda(t)
    return t.data_ptr(), t.numel() * t.element_size()


def _opt_ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def _dtype(x: torch.Tensor, name: str) -> int:
    if x.dtype not in _DTYPES:
        raise TypeError(f"{name} must be bfloat16, float16 or float32, got {x.dtype}")
    return _DTYPES[x.dtype]


def _mask(active_mask: torch.Tensor | None, n: int) -> int | None:
    if active_mask is None:
        return None
    if active_mask.dtype not in (torch.bool, torch.uint8):
        raise TypeError("active_mask must be bool or uint8")
    if active_mask.dim() != 1 or active_mask.shape[0] != n or (n > 1 and active_mask.stride(0) != 1):
        raise ValueError(f"active_mask must be a contiguous [{n}] tensor")
    _cuda(active_mask)
    return active_mask.data_ptr()
