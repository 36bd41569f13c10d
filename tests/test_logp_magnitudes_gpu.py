"""The plain log-probability and its gradient in rows of large logits and at small temperatures,
where FP32 (and from 2^53 on 64 bits) has no digits left for log S beside the maximum: against
the definition in 64 bits, which takes the maximum off first.

Tolerances, u = 2^-24: S is within 1e-5 (as the forward's other tests have it); the backward's lp =
(s x - lse) - lse_lo is off by a rounding of each of three numbers below 2^-24 |lse| + 25 and by
what lse_lo leaves of LSE, 2^-49 |lse|: together 2^-46 |lse| + 75 u.  At temperature 1 the first
is exact, both are FP32 numbers next to one another."""

import pytest
import torch

import selected_token_logprob_gb300 as flp
from test_logp_topk_gpu import HALF, TINY, close, exact, exact_grad
from test_logp_topk_magnitudes_gpu import TYPES, U, build, held

pytestmark = pytest.mark.gpu
CASES = [(kind, 1.0) for kind in ("neighbours", "lowest and inf", "large and inf", "halves", "filled")] + \
    [("ordinary", 1e-8), ("ordinary", 3e-7), ("ordinary", 2e-5), ("ordinary", 1e-3), ("ordinary", 0.7)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("v", [40, 5000, 151936])
@pytest.mark.parametrize("kind,temperature", CASES)
def test_forward_and_backward(kind, temperature, v, dtype):
    g = torch.Generator(device="cuda").manual_seed(v + len(kind))
    x = build(kind, v, dtype, g)
    n = x.shape[0]
    y = x.float().argmax(1)
    other = torch.randint(0, v, (n,), generator=g, device="cuda")
    y = torch.where((torch.arange(n, device="cuda") % 5 == 0) & x.gather(1, other[:, None])[:, 0].isfinite(), other, y)
    y[3] = -100
    grad = torch.randn(n, generator=g, device="cuda") * temperature
    kw = dict(temperature=temperature)
    logp, lse, lo = flp.fused_logp_forward(x, y, with_lse_lo=True, **kw)
    e = exact(x, y, 1, temperature)
    s = float(torch.tensor(1 / temperature, dtype=torch.float32))
    held(logp, e["logp"])
    z = torch.logsumexp(x.double() * s, 1)
    close(lse, z, 1.2e-5 + U * z.abs())
    want, size = exact_grad(e, y, grad, None, None, temperature)
    lp_off = 75 * U + (0 if temperature == 1.0 else 2.0 ** -46 * z.abs()[:, None])
    tol = want.abs() * HALF[dtype] + TINY[dtype] + size * (4e-5 + lp_off) + 2.0 ** -126 * s * grad.abs().double()[:, None]
    got = flp.fused_logp_backward(x, y, lse, grad, lse_lo=lo, **kw)
    close(got, want, tol)
    # in place, rows of another alignment, and the vocabulary's shards give the same bits
    own = x.clone()
    flp.fused_logp_backward(own, y, lse, grad, dlogits=own, lse_lo=lo, **kw)
    assert torch.equal(own, got)
    buf = torch.full((n * (v + 3) + 8,), 5.0, dtype=dtype, device="cuda")
    out = buf[1:1 + n * (v + 3)].view(n, v + 3)[:, :v]
    flp.fused_logp_backward(x, y, lse, grad, dlogits=out, lse_lo=lo, **kw)
    assert torch.equal(out, got)
    out.fill_(5.0)
    assert bool((buf == 5.0).all())
    w = flp.flp_tile_width(v)
    cut = min(v, 3 * w)
    pm, ps = (torch.zeros((n, 16), device="cuda") for _ in range(2))
    pm.fill_(-float("inf"))
    sel = torch.zeros(n, device="cuda")
    for a, b in ((0, cut), (cut, v)):
        if b > a:
            part = x[:, a:b].contiguous()
            flp.logp_shard_partials(part, a, b - a, v, y, pm, ps, sel, **kw)
            d = flp.logp_shard_backward(part, a, b - a, v, y, lse, grad, lse_lo=lo, **kw)
            assert torch.equal(d, got[:, a:b])
    merged = flp.logp_merge_partials(pm, ps, sel, y, v, with_lse_lo=True, **kw)
    on = e["active"]
    for p, q in zip(merged, (logp, lse, lo)):
        assert torch.equal(p[on], q[on])
    assert flp.flp_device_error(0) == 0
