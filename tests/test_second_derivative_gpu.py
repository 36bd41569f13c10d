"""GPU test: a second derivative through the norm's autograd function is refused."""

import pytest
import torch

import selected_token_logprob_gb300 as flp

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("center", [False, True])
def test_second_derivatives_are_refused(center):
    flp._lib.load(build_if_missing=True)
    g = torch.Generator(device=DEV).manual_seed(0)
    x = torch.randn(6, 64, device=DEV, generator=g).bfloat16().requires_grad_()
    w = torch.ones(64, device=DEV, requires_grad=True)
    y = flp.fused_layer_norm(x, w, center=center)
    made = torch.autograd.grad(y.float().square().sum(), (x, w), create_graph=True, retain_graph=True)
    first = torch.autograd.grad(y.float().square().sum(), (x, w))
    for m, f in zip(made, first):
        assert torch.equal(m, f)
        with pytest.raises(RuntimeError, match="differentiate twice"):
            (m.float().sum() + x.float().sum()).backward(retain_graph=True)
