"""Log-probabilities with entropy and alternatives where a logit's distance from the maximum is
lost beside the logit itself: large logits, small temperatures, closed columns of the type's
lowest number or -inf; against the definition in 64 bits, which takes the maximum off first.
Tolerances are those of test_logp_topk_gpu: they hold for a row's distances from its maximum,
whatever the maximum is."""

import math

import pytest
import torch

import selected_token_logprob_gb300 as flp
from test_logp_topk_gpu import HALF, TINY, close, exact, exact_grad

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16, torch.float32]
U = 2.0 ** -24


def build(kind, v, dtype, g):
    """24 rows: the open columns' values, the rest."""
    n, low = 24, torch.finfo(dtype).min
    x = torch.full((n, v), -math.inf, device="cuda", dtype=dtype)
    few = torch.rand((n, v), generator=g, device="cuda") < 0.02
    few[:, torch.randint(0, v, (1,), generator=g, device="cuda")] = True
    r = torch.randn((n, v), generator=g, device="cuda")
    if kind == "neighbours":         # one maximum of +-1e10 or so, half of it and less elsewhere
        top = 1e10 if dtype != torch.float16 else 6e4
        x = (r * 1e9 / 1e10 * top).clamp(-0.5 * top, 0.5 * top).to(dtype)
        x[:, v // 3] = top
        x[1::2] = -x[1::2].abs() - (top * 0.01 if dtype == torch.float16 else top)
    elif kind == "lowest and inf":   # few columns at the lowest number, the rest closed
        x[few] = low
    elif kind == "large and inf":    # few columns at one large value, the rest closed
        x[few] = -6e4 if dtype == torch.float16 else -1e10
    elif kind == "halves":           # two large values mixed
        x[:] = low / -4
        x[few] = low / -8
        x[::3] = -x[::3]
    elif kind == "filled":           # closed by a finite fill, all of a row or all but a few
        fill = [-1e4 if dtype == torch.float16 else -1e9, -6e4 if dtype == torch.float16 else -1e10, low]
        for i in range(n):
            x[i] = fill[i % 3]
        x[12:][few[12:]] = r[12:][few[12:]].to(dtype)
    else:                            # ordinary ones
        x = (r * 3).to(dtype)
        x[::4, ::2] = -math.inf
    return x


CASES = [(kind, 1.0) for kind in ("neighbours", "lowest and inf", "large and inf", "halves", "filled")] + \
    [("lowest and inf", 0.7), ("halves", 0.7), ("filled", 0.7), ("neighbours", 1.3),
     ("ordinary", 1e-9), ("ordinary", 3e-7), ("ordinary", 2e-5), ("ordinary", 1e-3), ("ordinary", 1e4), ("ordinary", 1e30)]


def case(kind, temperature, v, dtype):
    g = torch.Generator(device="cuda").manual_seed(v + len(kind))
    x = build(kind, v, dtype, g)
    k = min(v, 12)
    y = x.float().argmax(1)
    y[::5] = torch.randint(0, v, (len(y[::5]),), generator=g, device="cuda")
    y[3] = -100
    r = flp.fused_logp_topk_forward(x, y, k, temperature=temperature)
    torch.cuda.synchronize()
    assert flp.flp_device_error(0) == 0
    return x, y, r, exact(x, y, k, temperature), g


def held(got, want):
    """Log-probabilities, which are -inf where FP32 has no number for them (below -3.4028235e38)."""
    close(got, want.float().double(), 1.2e-5 * (1 + want.abs()))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("v", [40, 5000, 151936])
@pytest.mark.parametrize("kind,temperature", CASES)
def test_entropy_and_alternatives(kind, temperature, v, dtype):
    x, y, r, e, _ = case(kind, temperature, v, dtype)
    close(r.entropy, e["h"], 2e-5 * (1 + e["h"].abs()))
    assert torch.equal(r.top_ids, e["ids"])
    held(r.top_logp, e["top"])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("v", [40, 5000, 151936])
@pytest.mark.parametrize("kind,temperature", CASES)
def test_logp_and_lse(kind, temperature, v, dtype):
    x, y, r, e, _ = case(kind, temperature, v, dtype)
    held(r.logp, e["logp"])
    z = x.double() * float(torch.tensor(1 / temperature, dtype=torch.float32))
    lse = torch.where(e["active"], torch.logsumexp(z, 1), 0)
    in_range = lse.float().isfinite()
    close(r.lse[in_range], lse[in_range], (1.2e-5 + U * lse.abs())[in_range])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("v", [4000, 151936])
def test_a_nan_in_a_closed_tile(v, dtype):
    """A row's NaN makes its results NaN wherever it lies: 8 columns a lane of a warp and step,
    beside closed columns alone, with open ones in another place of the row or nowhere."""
    lanes = [0, 5, 16, 31]
    x = torch.full((2 * len(lanes) + 1, v), -math.inf, device="cuda", dtype=dtype)
    for i, lane in enumerate(lanes):
        x[2 * i, v // 2 // 256 * 256 + 8 * lane + i] = math.nan
        x[2 * i + 1] = x[2 * i]
        x[2 * i + 1, 3:9] = 1.0      # open
    x[-1, 3:9] = 1.0
    y = torch.full((x.shape[0],), 4, device="cuda")
    r = flp.fused_logp_topk_forward(x, y, 3)
    for t in (r.logp, r.lse, r.entropy, r.top_logp[:, 0]):
        assert bool(t[:-1].isnan().all()), t
    assert bool(x.float().isnan().gather(1, r.top_ids[:, :1])[:-1].all())
    assert abs(r.logp[-1].item() + math.log(6)) <= 2e-5 and abs(r.entropy[-1].item() - math.log(6)) <= 6e-5


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("v", [40, 5000, 151936])
@pytest.mark.parametrize("kind,temperature", CASES)
def test_backward(kind, temperature, v, dtype):
    x, y, r, e, g = case(kind, temperature, v, dtype)
    n, k = r.top_ids.shape
    s = float(torch.tensor(1 / temperature, dtype=torch.float32))
    gl = torch.randn(n, generator=g, device="cuda") / s
    gh = torch.rand(n, generator=g, device="cuda") / s
    gt = torch.rand((n, k), generator=g, device="cuda") / s
    for up in ((gl, gh, gt), (gl, None, None), (None, gh, None), (None, None, gt)):
        want, size = exact_grad(e, y, *up, temperature=temperature)
        # as there; the factors lp + H count for |lp| <= 88 (p is 0 below)
        tol = want.abs() * HALF[dtype] + TINY[dtype] + size * 2e-5 * (88 if up[1] is not None else 2)
        # p below 2^-126 is flushed to 0: off by that times the factor s (G + gh (lp + H)) beside it
        factor = sum(0 if u is None else (u if u.dim() == 1 else u.sum(1)).abs() for u in (up[0], up[2]))
        if up[1] is not None:
            factor = factor + up[1] * (88 + e["h"])
        tol = tol + 2.0 ** -126 * s * factor.double()[:, None]
        got = flp.fused_logp_topk_backward(x, y, r, *up, temperature=temperature)
        close(got, want, tol)
        own = x.clone()
        assert flp.fused_logp_topk_backward(own, y, r, *up, temperature=temperature, dlogits=own) is own
        assert torch.equal(own, got)
        # rows of another alignment
        buf = torch.full((n * (v + 3) + 8,), 5.0, dtype=dtype, device="cuda")
        out = buf[1:1 + n * (v + 3)].view(n, v + 3)[:, :v]
        flp.fused_logp_topk_backward(x, y, r, *up, temperature=temperature, dlogits=out)
        assert torch.equal(out, got)
        out.fill_(5.0)
        assert bool((buf == 5.0).all())
