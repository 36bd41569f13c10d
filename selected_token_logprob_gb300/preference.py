"""Preference loss of packed pairs of sequences on the selected-token logp."""

from __future__ import annotations

import ctypes
import functools

import torch

from . import _lib
from ._args import _cuda, _mask, _opt_ptr, _stream, _vec, _workspace

PREFERENCE_KINDS = {"sigmoid": 0, "hinge": 1, "ipo": 2}
PREFERENCE_LAYOUTS = {"interleaved": 0, "halves": 1}


def logp_preference_loss(logp: torch.Tensor, cu_seqlens: torch.Tensor, ref_logp: torch.Tensor | None = None,
                         active_mask: torch.Tensor | None = None, kind: str = "sigmoid", beta: float = 0.1,
                         label_smoothing: float = 0.0, margin: float = 0.0, average: bool = False,
                         layout: str = "interleaved", normalizer: float = 0.0,
                         workspace: torch.Tensor | None = None):
    """Preference loss of pairs of packed sequences: (loss FP32 [1], grad FP32
    [N] = d loss / d logp, rewards FP32 [P, 2] = beta times each pair's chosen
    and rejected log-ratio).  ``grad`` is the upstream gradient for
    ``fused_logp_backward`` and ``fused_linear_logp_backward``.

    Sequence s is tokens [cu_seqlens[s], cu_seqlens[s + 1]) of the packed logp;
    pair p is sequences (2p, 2p + 1) as (chosen, rejected) with ``layout``
    "interleaved", or (p, p + P) with "halves".  Its log-ratio is the sum (the
    mean with ``average``) of logp - ref_logp over the active tokens.  kind:
    "sigmoid" (with ``label_smoothing`` and ``margin``), "hinge" or "ipo".  The
    loss is the mean over the pairs whose sides both have an active token, or
    their sum over ``normalizer`` when that is positive.  ``workspace`` (a CUDA
    byte tensor of logp_preference_loss_workspace_size(N, S) bytes) is
    allocated when not given."""
    if kind not in PREFERENCE_KINDS:
        raise ValueError(f"kind must be one of {sorted(PREFERENCE_KINDS)} (got {kind!r})")
    if layout not in PREFERENCE_LAYOUTS:
        raise ValueError(f"layout must be one of {sorted(PREFERENCE_LAYOUTS)} (got {layout!r})")
    n = logp.shape[0] if logp.dim() == 1 else -1
    _vec(logp, "logp", n, torch.float32)
    if ref_logp is not None:
        _vec(ref_logp, "ref_logp", n, torch.float32)
        _cuda(ref_logp)
    if cu_seqlens.dtype != torch.int64 or cu_seqlens.dim() != 1 or cu_seqlens.shape[0] % 2 != 1:
        raise ValueError("cu_seqlens must be an int64 [S + 1] tensor with an even number S of sequences")
    _cuda(logp, cu_seqlens)
    mp = _mask(active_mask, n)
    cu_seqlens = cu_seqlens.contiguous()
    nseq = cu_seqlens.shape[0] - 1
    dev = logp.device
    loss = torch.empty(1, dtype=torch.float32, device=dev)
    grad = torch.empty(n, dtype=torch.float32, device=dev)
    rewards = torch.empty((nseq // 2, 2), dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = torch.empty(logp_preference_loss_workspace_size(n, nseq), dtype=torch.uint8, device=dev)
    wptr, wbytes = _workspace(workspace)
    st = _lib.load().logp_preference_loss(
        logp.data_ptr(), _opt_ptr(ref_logp), mp, cu_seqlens.data_ptr(), nseq, n, PREFERENCE_KINDS[kind],
        PREFERENCE_LAYOUTS[layout], 1 if average else 0, beta, label_smoothing, margin, normalizer,
        wptr, wbytes, loss.data_ptr(), grad.data_ptr(), rewards.data_ptr(), _stream(logp))
    _lib.check("logp_preference_loss", st)
    return loss, grad, rewards


@functools.lru_cache(maxsize=256)
def logp_preference_loss_workspace_size(n: int, num_seqs: int) -> int:
    """Bytes of device scratch that logp_preference_loss needs."""
    b = ctypes.c_int64(0)
    _lib.check("logp_preference_loss_workspace_size",
               _lib.load().logp_preference_loss_workspace_size(int(n), int(num_seqs), ctypes.byref(b)))
    return int(b.value)
