"""The preference-tuning step of examples/preference_step.py, all operators
together: its gradients against the same chain in 64 bits, and a few steps of
training.

Tolerance of the gradients: the chain rounds to BF16 at h, y, dZ (inside the LM
head's backward), dh and the final product, each at most 2^-9 of a value in
random directions; the norms of the differences stay within 5 * 2^-9 * 2 of the
gradient's norm (the factor 2 for the softmax's and the norm's gain on y's
error), 2e-2."""

import importlib.util
import os

import pytest
import torch

import selected_token_logprob_gb300 as flp

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def step():
    flp._lib.load(build_if_missing=True)
    spec = importlib.util.spec_from_file_location("preference_step", os.path.join(ROOT, "examples", "preference_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_gradients_against_64_bits(step):
    hidden, lm_head, targets, cu, mask = step.synthetic(pairs=6, mean_len=30)
    g = torch.Generator(device="cuda").manual_seed(1)
    d = hidden.shape[1]
    proj = (torch.randn(d, d, generator=g, device="cuda") * 0.3 / d ** 0.5).bfloat16()
    w = 1 + 0.1 * torch.randn(d, generator=g, device="cuda")
    ref = -torch.rand(hidden.shape[0], generator=g, device="cuda") - 6.5
    loss, rewards, dp, dw = step.gradients(hidden, proj, w, lm_head, targets, cu, mask, ref, beta=0.2)

    P, W = proj.double().requires_grad_(), w.double().requires_grad_()
    H = hidden.double()
    h = H + H @ P.T
    y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + step.EPS) * W
    logp = torch.log_softmax(y @ lm_head.double().T, 1).gather(1, targets[:, None])[:, 0]
    diff = torch.where(mask, logp - ref.double(), 0.0)
    r = torch.stack([diff[cu[s]:cu[s + 1]].sum() for s in range(len(cu) - 1)])
    want = torch.nn.functional.softplus(-0.2 * (r[0::2] - r[1::2])).mean()
    want.backward()
    assert abs(loss.item() - want.item()) <= 2e-2 * want.item()
    for got, exact in ((dp, P.grad), (dw, W.grad)):
        assert (got.double() - exact).norm() <= 2e-2 * exact.norm()


def test_training_wins_the_pairs(step, capsys):
    step.main(steps=12)
    lines = capsys.readouterr().out.strip().splitlines()
    loss = [float(x.split("loss")[1].split()[0]) for x in lines]
    won = float(lines[-1].split("won")[1])
    assert abs(loss[0] - 0.6931) < 1e-3      # the policy starts at the reference
    assert loss[-1] < 0.5 * loss[0] and won == 1.0
    assert flp.flp_device_error(0) == 0
