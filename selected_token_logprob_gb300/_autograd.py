"""What the autograd functions of the package share."""

from __future__ import annotations

import torch


class _Once(torch.autograd.Function):
    """Its first inputs (``count`` of them) as they are; the others only give it a graph,
    in which nothing can be differentiated."""

    @staticmethod
    def forward(ctx, count, *tensors):
        out = tuple(t.detach() for t in tensors[:count])
        return out if count > 1 else out[0]

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError("trying to differentiate twice a function whose gradients have no derivative here")


def once(grads: tuple, *inputs) -> tuple:
    """``grads`` (tensors or None) of a backward that depends on ``inputs``.  The kernels
    record no graph; under create_graph the gradients get one that refuses a second
    derivative, which would otherwise miss what goes through them without a word.
    (torch's once_differentiable looks at the incoming gradient alone.)"""
    if not torch.is_grad_enabled():
        return grads
    given = [g for g in grads if g is not None]
    made = _Once.apply(len(given), *given, *[t for t in inputs if t is not None])
    made = iter(made if isinstance(made, tuple) else (made,))
    return tuple(None if g is None else next(made) for g in grads)
