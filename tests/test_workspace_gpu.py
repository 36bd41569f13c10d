"""GPU tests of what the calls take as scratch: enough bytes that the tensor owns.

An expanded tensor counts more elements than it has memory, so it must be refused
before any launch (nothing here writes past an allocation)."""

import pytest
import torch

import selected_token_logprob_gb300 as flp

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    flp._lib.load(build_if_missing=True)


def _norm_backward(ws):
    x = torch.randn(9, 64, device=DEV, generator=torch.Generator(device=DEV).manual_seed(0))
    _, mean, rstd = flp.fused_layer_norm_forward(x)
    return flp.fused_layer_norm_backward(x, x, None, mean, rstd, workspace=ws)


def _preference(ws):
    logp = -torch.arange(1.0, 11.0, device=DEV)
    return flp.logp_preference_loss(logp, torch.tensor([0, 4, 10], device=DEV), workspace=ws)


def _orthogonalize(ws):
    return flp.orthogonalize(torch.randn(20, 30, device=DEV, generator=torch.Generator(device=DEV).manual_seed(1)),
                             workspace=ws)


def _grpo(ws):
    logp = -torch.arange(1.0, 11.0, device=DEV)
    return flp.logp_grpo_loss(logp, logp + 0.1, torch.ones(10, device=DEV), workspace=ws)


def _linear(ws):
    g = torch.Generator(device=DEV).manual_seed(2)
    h = torch.randn(8, 64, device=DEV, generator=g).bfloat16()
    w = torch.randn(512, 64, device=DEV, generator=g).bfloat16()
    return flp.fused_linear_logp_forward(h, w, torch.arange(8, device=DEV), workspace=ws)


@pytest.mark.parametrize("call", [_norm_backward, _preference, _orthogonalize, _grpo, _linear])
def test_scratch_must_be_the_callers_own_bytes(call):
    want = call(None)
    size = 8 << 20
    for ws in (torch.empty(1, dtype=torch.uint8, device=DEV).expand(size),
               torch.empty(2 * size, dtype=torch.uint8, device=DEV)[::2]):
        with pytest.raises(ValueError, match="contiguous"):
            call(ws)
    got = call(torch.full((size,), 255, dtype=torch.uint8, device=DEV))
    for a, b in zip(got, want):
        assert a is b is None or torch.equal(a, b)
