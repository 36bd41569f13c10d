"""The fused LM head's gradients into wider buffers: what lies behind their last column stays, where
that column ends inside 16 bytes of a row that starts on such a boundary, too."""

import pytest
import torch

import selected_token_logprob_gb300 as flp

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,d,v", [(300, 130, 700), (5000, 133, 300), (260, 519, 1500), (300, 128, 700)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_columns_behind(n, d, v, accumulate):
    g = torch.Generator(device="cuda").manual_seed(n + d)

    def operand(rows):
        return torch.randn((rows, -(-d // 8) * 8), generator=g, device="cuda").bfloat16()[:, :d]

    h, w = operand(n), operand(v) * 0.1
    w = torch.nn.functional.pad(w, (0, -d % 8))[:, :d]
    y = torch.randint(0, v, (n,), generator=g, device="cuda")
    up = torch.randn(n, generator=g, device="cuda")
    _, lse, lo = flp.fused_linear_logp_forward(h, w, y, with_lse_lo=True)
    start = torch.randn((v, d), generator=g, device="cuda")
    kw = dict(lse_lo=lo, accumulate_dweight=accumulate)
    want_h, want_w = flp.fused_linear_logp_backward(h, w, y, lse, up, dweight=start.clone(), **kw)
    ld = -(-d // 4) * 4 + 4
    bufs = [torch.full((rows * ld + 16,), 7.0, device="cuda") for rows in (n, v)]
    dh, dw = (b[:rows * ld].view(rows, ld)[:, :d] for b, rows in zip(bufs, (n, v)))
    dw.copy_(start)
    flp.fused_linear_logp_backward(h, w, y, lse, up, dhidden=dh, dweight=dw, **kw)
    assert torch.equal(dh, want_h) and torch.equal(dw, want_w)
    for t, b in ((dh, bufs[0]), (dw, bufs[1])):
        t.fill_(7.0)
        assert bool((b == 7.0).all())
    assert flp.flp_device_error(0) == 0
