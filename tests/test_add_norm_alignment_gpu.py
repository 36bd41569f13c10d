"""Residual addition and RMS norm: the bits of a row depend on the row alone, wherever its
tensors lie (each of them on and off 16-byte boundaries), forward and backward."""

import pytest
import torch

import selected_token_logprob_gb300 as flp

pytestmark = pytest.mark.gpu


def at(t, lead, pad):
    """t's values in a buffer, `lead` elements in and in rows `pad` wider."""
    n, d = t.shape
    buf = torch.zeros(lead + n * (d + pad) + 16, dtype=t.dtype, device="cuda")
    return buf[lead:lead + n * (d + pad)].view(n, d + pad)[:, :d].copy_(t)


@pytest.mark.parametrize("d", [64, 104, 256, 512, 1024, 2048, 4096, 8192, 8200, 16384, 20000])
@pytest.mark.parametrize("dtype,wide_dy", [(torch.bfloat16, False), (torch.bfloat16, True), (torch.float16, True),
                                           (torch.float32, True)])
def test_bits_do_not_depend_on_the_place(d, dtype, wide_dy):
    g = torch.Generator(device="cuda").manual_seed(d)
    n = 61
    x, r, dh = (torch.randn((n, d), generator=g, device="cuda").to(dtype) for _ in range(3))
    dy = torch.randn((n, d), generator=g, device="cuda").to(torch.float32 if wide_dy else dtype)
    w = 1 + 0.3 * torch.randn(d, generator=g, device="cuda")
    for quantize in (False, True):
        want = flp.fused_add_rms_norm_forward(x, r, w, quantize=quantize)
        for place in range(3):
            t = [at(v, 1, 0) if place == i else at(v, 0, 3) if place == i + 1 else v for i, v in enumerate((x, r))]
            got = flp.fused_add_rms_norm_forward(*t, w, quantize=quantize)
            assert torch.equal(got.h, want.h) and torch.equal(got.rstd, want.rstd)
            assert torch.equal(got.y.contiguous().view(torch.uint8), want.y.contiguous().view(torch.uint8))
            assert not quantize or torch.equal(got.scale, want.scale)
    for add in (dh, None):
        dx, _ = flp.fused_add_rms_norm_backward(dy, add, want.h, w, want.rstd)
        for which in range(4):
            for lead, pad in ((1, 0), (0, 1)):
                t = [v if v is None or i != which else at(v, lead, pad) for i, v in enumerate((dy, add, want.h, dx))]
                got, _ = flp.fused_add_rms_norm_backward(t[0], t[1], t[2], w, want.rstd, dx=t[3].clone(
                    memory_format=torch.preserve_format) if which != 3 else t[3].zero_())
                assert torch.equal(got, dx), (which, lead, pad)
