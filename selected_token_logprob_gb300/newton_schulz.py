"""Newton-Schulz orthogonalisation of a weight's update on the tensor cores."""

from __future__ import annotations

import ctypes
import functools

import torch

from . import _lib
from ._args import _DTYPES, _cuda, _dtype, _stream, _workspace

#: (a, b, c) of the usual quintic step X <- a X + (b A + c A^2) X, A = X X^T.
ORTHOGONALIZE_COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def _matrices(x: torch.Tensor, name: str):
    """(batch, rows, cols, ld, stride) of a 2-D or 3-D tensor whose rows are
    contiguous."""
    if x.dim() not in (2, 3):
        raise ValueError(f"{name} must be [M, N] or [B, M, N], got shape {tuple(x.shape)}")
    batch = x.shape[0] if x.dim() == 3 else 1
    rows, cols = x.shape[-2:]
    if cols > 1 and x.stride(-1) != 1:
        raise ValueError(f"{name} rows must be contiguous (stride(-1) == 1)")
    ld = x.stride(-2) if rows > 1 else max(cols, x.stride(-2))
    if x.numel() and ld < cols:
        raise ValueError(f"{name} row stride {ld} is smaller than its width {cols}")
    return batch, rows, cols, max(ld, cols), (x.stride(0) if x.dim() == 3 else 0)


def orthogonalize(x: torch.Tensor, steps: int = 5, coefficients=ORTHOGONALIZE_COEFFICIENTS, eps: float = 1e-7,
                  scale: float = 1.0, out: torch.Tensor | None = None, out_dtype: torch.dtype = torch.bfloat16,
                  workspace: torch.Tensor | None = None) -> torch.Tensor:
    """``scale`` times the Newton-Schulz orthogonalisation of x [M, N], or of
    every matrix of a stack x [B, M, N] (BF16, FP16 or FP32): X = x / (|x|_F +
    eps), then ``steps`` times X <- a X + (b A + c A^2) X with A = X X^T on the
    smaller side.  ``coefficients`` is one (a, b, c) or one per step.  Returns
    ``out`` (BF16, the default ``out_dtype``, or FP32), which may be x.  The
    products run on FP16 operands with compensated carries: five of the usual
    steps are within 3e-4 to 2e-3 of the result's norm of the exact one (4e-3 at
    most, 1e-2 where a side is below 8), six within 4.5e-3; more steps lose more where singular values are near
    zero (eight 1.5e-2, ten 8e-2).  ``workspace`` (a CUDA byte
    tensor of orthogonalize_workspace_size(B, M, N) bytes) is allocated when
    not given."""
    batch, rows, cols, ld, stride = _matrices(x, "x")
    dt = _dtype(x, "x")
    steps = int(steps)
    flat = list(coefficients)
    if len(flat) == 3 and not hasattr(flat[0], "__len__"):
        flat = [tuple(flat)] * steps
    if steps < 1 or len(flat) != steps or any(len(t) != 3 for t in flat):
        raise ValueError("coefficients must be one (a, b, c) or one per step, and steps >= 1")
    if out is None:
        out = torch.empty(x.shape, dtype=out_dtype, device=x.device)
    if out.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"out must be bfloat16 or float32, got {out.dtype}")
    if out.shape != x.shape:
        raise ValueError(f"out must have x's shape {tuple(x.shape)}, got {tuple(out.shape)}")
    _, _, _, ld_out, stride_out = _matrices(out, "out")
    _cuda(x, out)
    if x.numel() == 0:
        return out
    if workspace is None:
        workspace = torch.empty(orthogonalize_workspace_size(batch, rows, cols), dtype=torch.uint8, device=x.device)
    wptr, wbytes = _workspace(workspace)
    coef = (ctypes.c_float * (3 * steps))(*[float(v) for t in flat for v in t])
    st = _lib.load().flp_orthogonalize(
        x.data_ptr(), dt, batch, rows, cols, ld, stride, steps, coef, float(eps), float(scale), wptr, wbytes,
        out.data_ptr(), _DTYPES[out.dtype], ld_out, stride_out,
        _stream(x))
    _lib.check("flp_orthogonalize", st)
    return out


@functools.lru_cache(maxsize=256)
def orthogonalize_workspace_size(batch: int, rows: int, cols: int) -> int:
    """Bytes of device scratch that orthogonalize needs."""
    b = ctypes.c_int64(0)
    _lib.check("flp_orthogonalize_workspace_size",
               _lib.load().flp_orthogonalize_workspace_size(int(batch), int(rows), int(cols), ctypes.byref(b)))
    return int(b.value)
