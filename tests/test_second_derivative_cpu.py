"""The norm's autograd function returns gradients without a graph of their own, so a
second derivative through them has to be refused, not left out.  The kernels are
replaced by host stand-ins here; tests/test_second_derivative_gpu.py runs them."""

import pytest
import torch

import selected_token_logprob_gb300 as flp
from selected_token_logprob_gb300 import norm as norm_module


@pytest.fixture(autouse=True)
def _host(monkeypatch):
    monkeypatch.setattr(norm_module, "fused_layer_norm_forward",
                        lambda x, w, b, eps, center: (x.detach() * 2, x.detach()[:, 0], x.detach()[:, 0]))
    monkeypatch.setattr(norm_module, "fused_layer_norm_backward",
                        lambda dy, x, w, *a, with_dweight, with_dbias, **k: (
                            dy.detach() * 2, torch.ones(4) if with_dweight else None,
                            torch.ones(4) if with_dbias else None))


@pytest.mark.parametrize("vectors", [0, 1, 2])
def test_second_derivatives_are_refused(vectors):
    ins = [torch.randn(3, 4, requires_grad=True)] + [torch.randn(4, requires_grad=True) for _ in range(vectors)]
    grads = torch.autograd.grad(flp.fused_layer_norm(*ins).sum(), ins, create_graph=True)
    assert torch.equal(grads[0], torch.full((3, 4), 2.0)) and len(grads) == 1 + vectors
    for g in grads:
        with pytest.raises(RuntimeError, match="differentiate twice"):
            (g.square().sum() + ins[0].square().sum()).backward(retain_graph=True)


def test_a_penalty_on_the_incoming_gradient_is_refused_too():
    x, s = torch.randn(3, 4), torch.ones((), requires_grad=True)
    x.requires_grad_()
    (g,) = torch.autograd.grad((flp.fused_layer_norm(x) * s).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="differentiate twice"):
        g.sum().backward()


def test_plain_backward_has_no_graph():
    x, w = torch.randn(3, 4, requires_grad=True), torch.ones(4, requires_grad=True)
    flp.fused_layer_norm(x, w).sum().backward()
    assert torch.equal(x.grad, torch.full((3, 4), 2.0)) and torch.equal(w.grad, torch.ones(4))
    assert not x.grad.requires_grad and not w.grad.requires_grad
