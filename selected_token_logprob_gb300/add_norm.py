"""RMS norm behind the residual's addition, with an output in the rows' type or
in 8 bits with scales; forward, backward, autograd."""

from __future__ import annotations

from typing import NamedTuple

import torch

from . import _lib
from ._args import _DTYPES, _cuda, _dtype, _opt_ptr, _rows, _stream, _vec, _workspace
from ._autograd import once
from .norm import _affine, _sum_output, fused_layer_norm_backward_workspace_size


class AddRmsNorm(NamedTuple):
    """What ``fused_add_rms_norm_forward`` returns."""

    y: torch.Tensor              # [N, D]: x's dtype, or float8_e4m3fn with scales
    scale: torch.Tensor | None   # FP32 [ceil(D / 128), N]; None unless quantised
    h: torch.Tensor              # [N, D]: x + residual (x itself without a residual)
    rstd: torch.Tensor           # FP32 [N]


def _like(t: torch.Tensor | None, name: str, x: torch.Tensor, dtype: torch.dtype):
    """Row stride of an output or second input of x's shape."""
    if t.dtype != dtype or t.shape != x.shape:
        raise ValueError(f"{name} must be a {dtype} tensor of x's shape {tuple(x.shape)}")
    _, _, ld = _rows(t, name)
    _cuda(t)
    return ld


def fused_add_rms_norm_forward(x: torch.Tensor, residual: torch.Tensor | None = None,
                               weight: torch.Tensor | None = None, eps: float = 1e-6, quantize: bool = False,
                               h: torch.Tensor | None = None, y: torch.Tensor | None = None,
                               scale: torch.Tensor | None = None, rstd: torch.Tensor | None = None) -> AddRmsNorm:
    """``AddRmsNorm`` of the rows of x [N, D]: h = x + residual in x's dtype
    (the new residual stream; may be ``residual`` or ``x``, in place), and y =
    h rstd weight, rstd = (mean(h^2) + eps)^-1/2.  With ``quantize`` y is
    float8_e4m3fn with one FP32 scale for each 128 columns of a row (``scale``
    [ceil(D / 128), N], as ``fp8_matmul`` reads it), else x's dtype.  weight
    [D] has x's dtype or FP32."""
    n, d, ld = _rows(x, "x")
    dt = _dtype(x, "x")
    wdt = _affine(weight, None, x, d)
    if not 0.0 <= eps < float("inf"):
        raise ValueError(f"eps must be finite and >= 0, got {eps}")
    _cuda(x)
    dev = x.device
    ld_r = ld_h = 0
    if residual is None:
        if h is not None:
            raise ValueError("h is written with a residual only")
    else:
        ld_r = _like(residual, "residual", x, x.dtype)
        if h is None:
            h, ld_h = torch.empty((n, d), dtype=x.dtype, device=dev), d
        else:
            ld_h = _like(h, "h", x, x.dtype)
    if quantize:
        if y is None:   # rows on 16-byte boundaries, as the product reads them
            ld_y = -(-d // 16) * 16
            y = torch.empty_strided((n, d), (ld_y, 1), dtype=torch.float8_e4m3fn, device=dev)
        else:
            ld_y = _like(y, "y", x, torch.float8_e4m3fn)
        blocks = -(-d // 128)
        if scale is None:
            scale, ld_s = torch.empty((blocks, n), dtype=torch.float32, device=dev), n
        elif scale.dtype != torch.float32 or scale.shape != (blocks, n) or (n > 1 and scale.stride(1) != 1):
            raise ValueError(f"scale must be an FP32 [{blocks}, {n}] tensor with contiguous rows")
        else:
            _cuda(scale)
            ld_s = max(n, scale.stride(0)) if blocks == 1 else scale.stride(0)
    else:
        if scale is not None:
            raise ValueError("scale is written with quantize only")
        if y is None:
            y, ld_y = torch.empty((n, d), dtype=x.dtype, device=dev), d
        else:
            ld_y = _like(y, "y", x, x.dtype)
        ld_s = 0
    if rstd is None:
        rstd = torch.empty(n, dtype=torch.float32, device=dev)
    else:
        _vec(rstd, "rstd", n, torch.float32)
        _cuda(rstd)
    if n > 0:
        out = (None, 0, y.data_ptr(), ld_y) if quantize else (y.data_ptr(), ld_y, None, 0)
        st = _lib.load().fused_add_rms_norm_forward(
            x.data_ptr(), dt, n, d, ld, _opt_ptr(residual), ld_r, _opt_ptr(weight), wdt, eps, _opt_ptr(h), ld_h, *out,
            _opt_ptr(scale), ld_s, rstd.data_ptr(), _stream(x))
        _lib.check("fused_add_rms_norm_forward", st)
    return AddRmsNorm(y, scale, x if h is None else h, rstd)


def fused_add_rms_norm_backward(dy: torch.Tensor, dh: torch.Tensor | None, h: torch.Tensor,
                                weight: torch.Tensor | None, rstd: torch.Tensor, with_dweight: bool = True,
                                dx: torch.Tensor | None = None, dweight: torch.Tensor | None = None,
                                accumulate: bool = False, workspace: torch.Tensor | None = None):
    """(dx [N, D] of h's dtype, dweight FP32 [D] or None): the gradient of x,
    which is also the residual's, for the upstream gradients dy of y (h's dtype
    or FP32) and dh of h (h's dtype, or None).  A quantised y hands its gradient
    straight through.  ``dx`` may be ``dh``; with ``accumulate`` the given
    ``dweight`` is added to."""
    n, d, ld = _rows(h, "h")
    dt = _dtype(h, "h")
    wdt = _affine(weight, None, h, d)
    if dy.dtype != h.dtype and dy.dtype != torch.float32:
        raise TypeError(f"dy must be {h.dtype} or torch.float32, got {dy.dtype}")
    ld_dy = _like(dy, "dy", h, dy.dtype)
    ld_dh = 0 if dh is None else _like(dh, "dh", h, h.dtype)
    _vec(rstd, "rstd", n, torch.float32)
    _cuda(h, rstd)
    dev = h.device
    if dx is None:
        dx, ld_dx = torch.empty((n, d), dtype=h.dtype, device=dev), d
    else:
        ld_dx = _like(dx, "dx", h, h.dtype)
    dweight = _sum_output("dweight", dweight, with_dweight, accumulate, d, dev)
    wptr, wbytes = None, 0
    if workspace is not None:
        wptr, wbytes = _workspace(workspace)
    elif n > 0 and with_dweight:
        wbytes = fused_layer_norm_backward_workspace_size(d, n)
        workspace = torch.empty(wbytes, dtype=torch.uint8, device=dev)
        wptr = workspace.data_ptr()
    st = _lib.load().fused_add_rms_norm_backward(
        dy.data_ptr(), _DTYPES[dy.dtype], ld_dy, _opt_ptr(dh), ld_dh, h.data_ptr(), dt, n, d, ld, _opt_ptr(weight), wdt,
        rstd.data_ptr(), wptr, wbytes, dx.data_ptr(), ld_dx, _opt_ptr(dweight), 1 if accumulate else 0, _stream(h))
    _lib.check("fused_add_rms_norm_backward", st)
    return dx, dweight


def _readable(t: torch.Tensor | None):
    """A gradient as the kernels read it: broadcast or transposed ones are copied."""
    if t is None:
        return None
    n, d = t.shape
    return t.contiguous() if (d > 1 and t.stride(1) != 1) or (n > 1 and t.stride(0) < d) else t


class FusedAddRmsNorm(torch.autograd.Function):
    """(y, h) = FusedAddRmsNorm.apply(x, residual, weight, eps); saves h, the
    weight and the rows' FP32 rstd."""

    @staticmethod
    def forward(ctx, x, residual, weight=None, eps=1e-6):
        r = fused_add_rms_norm_forward(x, residual, weight, eps=eps)
        ctx.save_for_backward(r.h, weight, r.rstd)
        ctx.set_materialize_grads(False)
        return r.y, r.h

    @staticmethod
    def backward(ctx, dy, dh):
        h, weight, rstd = ctx.saved_tensors
        residual = ctx.needs_input_grad[1]
        if dy is None:
            (dx,) = once((dh,), dh)
            return dx, dx if residual else None, None, None
        dx, dw = fused_add_rms_norm_backward(
            _readable(dy), _readable(dh), h, weight, rstd,
            with_dweight=weight is not None and ctx.needs_input_grad[2])
        dw = dw if dw is None else dw.to(weight.dtype)
        dx, dw = once((dx, dw), dy, dh, h, weight)
        return dx, dx if residual else None, dw, None


def fused_add_rms_norm(x: torch.Tensor, residual: torch.Tensor, weight: torch.Tensor | None = None,
                       eps: float = 1e-6):
    """Autograd-aware (y, h): h = x + residual and y its RMS norm; see
    ``fused_add_rms_norm_forward``."""
    return FusedAddRmsNorm.apply(x, residual, weight, eps)
