"""The norm in front of the LM head: layer norm or, with ``center=False``, RMS
norm; forward, backward with the weight's and bias's gradients, autograd."""

from __future__ import annotations

import ctypes
import functools

import torch

from . import _lib
from ._args import _DTYPES, _cuda, _dtype, _opt_ptr, _rows, _stream, _vec, _workspace
from ._autograd import once


def _affine(weight, bias, x, d: int) -> int:
    """The C dtype of weight and bias (x's when neither is given)."""
    first = weight if weight is not None else bias
    if first is None:
        return _DTYPES[x.dtype]
    dtype = first.dtype
    if dtype != x.dtype and dtype != torch.float32:
        raise TypeError(f"weight and bias must be {x.dtype} or torch.float32, got {dtype}")
    if weight is not None:
        _vec(weight, "weight", d, dtype)
        _cuda(weight)
    if bias is not None:
        _vec(bias, "bias", d, dtype)
        _cuda(bias)
    return _DTYPES[dtype]


def fused_layer_norm_forward(x: torch.Tensor, weight: torch.Tensor | None = None,
                             bias: torch.Tensor | None = None, eps: float = 1e-5, center: bool = True,
                             y: torch.Tensor | None = None, mean: torch.Tensor | None = None,
                             rstd: torch.Tensor | None = None):
    """(y [N, D] of x's dtype, mean FP32 [N] or None, rstd FP32 [N]) of the
    rows of x [N, D]: y = (x - mean) * rstd * weight + bias.  With
    ``center=False`` no mean is taken (RMS norm; mean is None).  weight and
    bias [D] have x's dtype or FP32.  ``y`` may be ``x`` (in place)."""
    n, d, ld = _rows(x, "x")
    dt = _dtype(x, "x")
    wdt = _affine(weight, bias, x, d)
    if not 0.0 <= eps < float("inf"):
        raise ValueError(f"eps must be finite and >= 0, got {eps}")
    _cuda(x)
    dev = x.device
    if y is None:
        y, ld_y = torch.empty((n, d), dtype=x.dtype, device=dev), d
    else:
        if y.dtype != x.dtype or y.shape != x.shape:
            raise ValueError("y must have x's dtype and shape")
        _, _, ld_y = _rows(y, "y")
        _cuda(y)
    if rstd is None:
        rstd = torch.empty(n, dtype=torch.float32, device=dev)
    else:
        _vec(rstd, "rstd", n, torch.float32)
        _cuda(rstd)
    if not center:
        mean = None
    elif mean is None:
        mean = torch.empty(n, dtype=torch.float32, device=dev)
    else:
        _vec(mean, "mean", n, torch.float32)
        _cuda(mean)
    if n > 0:
        st = _lib.load().fused_layer_norm_forward(
            x.data_ptr(), dt, n, d, ld, _opt_ptr(weight), _opt_ptr(bias), wdt, eps, 1 if center else 0,
            y.data_ptr(), ld_y, _opt_ptr(mean), rstd.data_ptr(), _stream(x))
        _lib.check("fused_layer_norm_forward", st)
    return y, mean, rstd


@functools.lru_cache(maxsize=256)
def fused_layer_norm_backward_workspace_size(d: int, n: int | None = None) -> int:
    """Bytes of device scratch that fused_layer_norm_backward needs for the
    partial sums of the weight's and bias's gradients: for ``n`` rows, or for
    any number of them."""
    b = ctypes.c_int64(0)
    if n is None:
        _lib.check("fused_layer_norm_backward_workspace_size",
                   _lib.load().fused_layer_norm_backward_workspace_size(int(d), ctypes.byref(b)))
    else:
        _lib.check("fused_layer_norm_backward_rows_workspace_size",
                   _lib.load().fused_layer_norm_backward_rows_workspace_size(int(n), int(d), ctypes.byref(b)))
    return int(b.value)


def _sum_output(name: str, t, wanted: bool, accumulate: bool, d: int, dev):
    if not wanted:
        return None
    if t is None:
        if accumulate:
            raise ValueError(f"accumulate needs the {name} tensor to add to")
        return torch.empty(d, dtype=torch.float32, device=dev)
    _vec(t, name, d, torch.float32)
    _cuda(t)
    return t


def fused_layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, weight: torch.Tensor | None,
                              mean: torch.Tensor | None, rstd: torch.Tensor, center: bool = True,
                              with_dweight: bool = True, with_dbias: bool = True,
                              dx: torch.Tensor | None = None, dweight: torch.Tensor | None = None,
                              dbias: torch.Tensor | None = None, accumulate: bool = False,
                              workspace: torch.Tensor | None = None):
    """(dx [N, D] of x's dtype, dweight FP32 [D], dbias FP32 [D]) of the norm
    for the upstream gradient dy [N, D] (x's dtype, or FP32 as
    ``fused_linear_logp_backward`` returns its dhidden), from the forward's
    mean and rstd.  dweight / dbias are None when not wanted; with
    ``accumulate`` the given ones are added to, not overwritten."""
    n, d, ld = _rows(x, "x")
    dt = _dtype(x, "x")
    wdt = _affine(weight, None, x, d)
    gdt = dy.dtype
    if gdt != x.dtype and gdt != torch.float32:
        raise TypeError(f"dy must be {x.dtype} or torch.float32, got {gdt}")
    if dy.shape != x.shape:
        raise ValueError(f"dy must have x's shape {(n, d)}, got {tuple(dy.shape)}")
    _, _, ld_dy = _rows(dy, "dy")
    _vec(rstd, "rstd", n, torch.float32)
    _cuda(dy, x, rstd)
    if not center:
        mean = None
    elif mean is None:
        raise ValueError("center=True needs the forward's mean")
    else:
        _vec(mean, "mean", n, torch.float32)
        _cuda(mean)
    dev = x.device
    if dx is None:
        dx, ld_dx = torch.empty((n, d), dtype=x.dtype, device=dev), d
    else:
        if dx.dtype != x.dtype or dx.shape != x.shape:
            raise ValueError("dx must have x's dtype and shape")
        _, _, ld_dx = _rows(dx, "dx")
        _cuda(dx)
    dweight = _sum_output("dweight", dweight, with_dweight, accumulate, d, dev)
    dbias = _sum_output("dbias", dbias, with_dbias, accumulate, d, dev)
    wptr, wbytes = None, 0
    if workspace is not None:
        wptr, wbytes = _workspace(workspace)
    elif n > 0 and (with_dweight or with_dbias):
        wbytes = fused_layer_norm_backward_workspace_size(d, n)
        workspace = torch.empty(wbytes, dtype=torch.uint8, device=dev)
        wptr = workspace.data_ptr()
    st = _lib.load().fused_layer_norm_backward(
        dy.data_ptr(), _DTYPES[gdt], ld_dy, x.data_ptr(), dt, n, d, ld, _opt_ptr(weight), wdt,
        _opt_ptr(mean), rstd.data_ptr(), 1 if center else 0, wptr, wbytes, dx.data_ptr(), ld_dx,
        _opt_ptr(dweight), _opt_ptr(dbias), 1 if accumulate else 0, _stream(x))
    _lib.check("fused_layer_norm_backward", st)
    return dx, dweight, dbias


class FusedLayerNorm(torch.autograd.Function):
    """y = FusedLayerNorm.apply(x, weight, bias, eps, center); saves x, the
    weight and the rows' FP32 statistics."""

    @staticmethod
    def forward(ctx, x, weight=None, bias=None, eps=1e-5, center=True):
        y, mean, rstd = fused_layer_norm_forward(x, weight, bias, eps=eps, center=center)
        ctx.save_for_backward(x, weight, mean, rstd)
        ctx.center = center
        ctx.bias_dtype = None if bias is None else bias.dtype
        return y

    @staticmethod
    def backward(ctx, dy):
        x, weight, mean, rstd = ctx.saved_tensors
        n, d = dy.shape
        if (d > 1 and dy.stride(1) != 1) or (n > 1 and dy.stride(0) < d):
            dy = dy.contiguous()   # a broadcast or transposed gradient
        dx, dw, db = fused_layer_norm_backward(
            dy, x, weight, mean, rstd, center=ctx.center,
            with_dweight=weight is not None and ctx.needs_input_grad[1],
            with_dbias=ctx.bias_dtype is not None and ctx.needs_input_grad[2])
        dw = dw if dw is None else dw.to(weight.dtype)
        db = db if db is None else db.to(ctx.bias_dtype)
        return *once((dx, dw, db), dy, x, weight), None, None


def fused_layer_norm(x: torch.Tensor, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None,
                     eps: float = 1e-5, center: bool = True) -> torch.Tensor:
    """Autograd-aware layer norm (RMS norm with ``center=False``) of the rows
    of x [N, D]."""
    return FusedLayerNorm.apply(x, weight, bias, eps, center)
