"""One preference-tuning step of a projection in front of the LM head, built from
this package's calls:

    h    = hidden + hidden @ projection.T
    y    = RMS norm of h                          fused_layer_norm_forward
    logp = selected-token logp of y @ lm_head.T   fused_linear_logp_forward
    loss, d loss / d logp                         logp_preference_loss
    dy   (FP32)                                   fused_linear_logp_backward
    dh, d norm weight                             fused_layer_norm_backward
    projection -= lr * orthogonalised momentum    orthogonalize

Run ``python examples/preference_step.py`` on a GB300: it tunes the projection
on synthetic pairs (the rejected answers shuffled) and prints the loss, the
reward margin and the share of pairs won.
"""

from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import selected_token_logprob_gb300 as flp  # noqa: E402

EPS = 1e-6


def forward(hidden, projection, norm_weight, lm_head, targets):
    """(logp, state for the backward) of the tuned head."""
    h = hidden + hidden @ projection.T
    y, _, rstd = flp.fused_layer_norm_forward(h, norm_weight, eps=EPS, center=False)
    logp, lse, lse_lo = flp.fused_linear_logp_forward(y, lm_head, targets, with_lse_lo=True)
    return logp, (h, y, rstd, lse, lse_lo)


def gradients(hidden, projection, norm_weight, lm_head, targets, cu_seqlens, mask, ref_logp, beta=0.1):
    """(loss, rewards, d projection FP32, d norm weight FP32) of one batch of pairs."""
    logp, (h, y, rstd, lse, lse_lo) = forward(hidden, projection, norm_weight, lm_head, targets)
    loss, dlogp, rewards = flp.logp_preference_loss(logp, cu_seqlens, ref_logp=ref_logp, active_mask=mask, beta=beta)
    dy, _ = flp.fused_linear_logp_backward(y, lm_head, targets, lse, dlogp, lse_lo=lse_lo)
    dh, dnorm, _ = flp.fused_layer_norm_backward(dy, h, norm_weight, None, rstd, center=False, with_dbias=False)
    return loss, rewards, (dh.T @ hidden).float(), dnorm


class OrthogonalSGD:
    """Momentum whose orthogonalised direction is the update of a matrix."""

    def __init__(self, like: torch.Tensor, lr: float, momentum: float = 0.95):
        self.buffer = torch.zeros(like.shape, dtype=torch.float32, device=like.device)
        self.lr, self.momentum = lr, momentum

    def step(self, parameter: torch.Tensor, grad: torch.Tensor) -> None:
        self.buffer.mul_(self.momentum).add_(grad)
        update = flp.orthogonalize(grad + self.momentum * self.buffer)   # Nesterov's look ahead
        parameter.sub_(update, alpha=self.lr)


def synthetic(pairs=24, mean_len=40, d=256, v=1000, seed=0, device="cuda"):
    """Hidden states, weights and packed pairs (chosen, rejected) of equal prompts."""
    g = torch.Generator(device="cpu").manual_seed(seed)
    lens = torch.randint(mean_len // 2, mean_len * 2, (2 * pairs,), generator=g)
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), torch.cumsum(lens, 0)])
    n = int(cu[-1])
    hidden = torch.randn(n, d, generator=g).bfloat16()
    lm_head = (torch.randn(v, d, generator=g) * 2 / d ** 0.5).bfloat16()
    targets = torch.randint(0, v, (n,), generator=g)
    mask = torch.rand(n, generator=g) > 0.2
    return [t.to(device) for t in (hidden, lm_head, targets, cu, mask)]


def main(steps: int = 20) -> None:
    hidden, lm_head, targets, cu, mask = synthetic()
    d = hidden.shape[1]
    projection = torch.zeros(d, d, dtype=torch.bfloat16, device=hidden.device)
    norm_weight = torch.ones(d, dtype=torch.float32, device=hidden.device)
    ref_logp, _ = forward(hidden, projection, norm_weight, lm_head, targets)
    optimiser = OrthogonalSGD(projection, lr=0.01)
    for k in range(steps):
        loss, rewards, dprojection, _ = gradients(hidden, projection, norm_weight, lm_head, targets, cu, mask, ref_logp)
        optimiser.step(projection, dprojection)
        margin = rewards[:, 0] - rewards[:, 1]
        print(f"step {k:2d}  loss {loss.item():.4f}  margin {margin.mean().item():+.4f}  "
              f"won {(margin > 0).float().mean().item():.2f}")


if __name__ == "__main__":
    main()
