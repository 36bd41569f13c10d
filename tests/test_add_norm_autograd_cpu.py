"""The autograd function of the norm behind the residual's addition without a residual, with either
output left out.  The kernels are replaced by host stand-ins; tests/test_add_norm_gpu.py runs them."""

import pytest
import torch

import selected_token_logprob_gb300 as flp
from selected_token_logprob_gb300 import add_norm as module


@pytest.fixture(autouse=True)
def _host(monkeypatch):
    def forward(x, residual=None, weight=None, eps=1e-6):
        h = x if residual is None else x.detach() + residual.detach()
        rstd = (h.detach().square().mean(1) + eps).rsqrt()
        return flp.AddRmsNorm(h.detach() * rstd[:, None] * (1 if weight is None else weight.detach()), None, h, rstd)

    def backward(dy, dh, h, weight, rstd, with_dweight=True):
        xh = h * rstd[:, None]
        g = dy * (1 if weight is None else weight)
        dx = rstd[:, None] * (g - xh * (g * xh).mean(1, keepdim=True)) + (0 if dh is None else dh)
        return dx, (dy * xh).sum(0) if with_dweight else None

    monkeypatch.setattr(module, "fused_add_rms_norm_forward", forward)
    monkeypatch.setattr(module, "fused_add_rms_norm_backward", lambda *a, **k: [
        None if t is None else t.detach() for t in backward(*a, **k)])


@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("use", ["y", "h", "both"])
def test_gradients(use, residual, weighted):
    gen = torch.Generator().manual_seed(0)
    x, r = (torch.randn((3, 5), generator=gen, dtype=torch.float64).requires_grad_() for _ in range(2))
    w = torch.randn(5, generator=gen, dtype=torch.float64).requires_grad_() if weighted else None
    a, b = (torch.randn((3, 5), generator=gen, dtype=torch.float64) for _ in range(2))
    a, b = (0 if use == "h" else a), (0 if use == "y" else b)

    def loss(y, h):
        return ((y * a).sum() if use != "h" else 0) + ((h * b).sum() if use != "y" else 0)

    leaves = [t for t in (x, r if residual else None, w) if t is not None]
    got = torch.autograd.grad(loss(*flp.fused_add_rms_norm(x, r if residual else None, w)), leaves, allow_unused=True)
    h = x + r if residual else x
    y = h * (h.square().mean(1, keepdim=True) + 1e-6).rsqrt() * (1 if w is None else w)
    want = torch.autograd.grad(loss(y, h), leaves, allow_unused=True)
    for p, q in zip(got, want):
        assert (p is None) == (q is None) and (p is None or torch.allclose(p, q, rtol=1e-12, atol=1e-14))


class _NoGradient(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x):
        return x * 1

    @staticmethod
    def backward(ctx, grad):
        return None


@pytest.mark.parametrize("create_graph", [False, True])
def test_no_gradient_comes_back(create_graph):
    x, r = (torch.randn((3, 5), dtype=torch.float64).requires_grad_() for _ in range(2))
    y, h = flp.fused_add_rms_norm(x, r)
    out = _NoGradient.apply(y).sum() + _NoGradient.apply(h).sum()
    assert torch.autograd.grad(out, (x, r), create_graph=create_graph, allow_unused=True) == (None, None)
