"""GPU test: a row's y, mean, rstd and dx depend on the row and the vectors alone, not on
where the rows lie.  Aligned and unaligned rows take different kernels, which add in the
same order, so the bits are the same at every width that either of them holds."""

import pytest
import torch

import selected_token_logprob_gb300 as flp

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _at(t, lead, pad):
    n, d = t.shape
    buf = torch.empty(n * (d + pad) + lead, dtype=t.dtype, device=DEV)
    v = buf[lead:].view(n, d + pad)[:, :d]
    v.copy_(t)
    return v


@pytest.mark.parametrize("d", [64, 128, 256, 512, 1024, 2048, 4096, 7992, 8008, 8192, 9216, 13992, 14016, 15000, 16384])
@pytest.mark.parametrize("dtype,wide_dy", [(torch.bfloat16, False), (torch.float16, True), (torch.float32, True)])
@pytest.mark.parametrize("center", [False, True])
def test_bits_do_not_depend_on_the_place(d, dtype, wide_dy, center):
    flp._lib.load(build_if_missing=True)
    g = torch.Generator(device=DEV).manual_seed(d)
    x = (torch.randn(9, d, generator=g, device=DEV) + 0.4).to(dtype)
    w = 1 + 0.2 * torch.randn(d, generator=g, device=DEV)
    dy = torch.randn(9, d, generator=g, device=DEV).to(torch.float32 if wide_dy else dtype)
    y, mean, rstd = flp.fused_layer_norm_forward(x, w, center=center)
    dx, _, _ = flp.fused_layer_norm_backward(dy, x, w, mean, rstd, center=center)
    for lead, pad in ((1, 1), (3, 8), (0, 5)):
        xs = _at(x, lead, pad)
        y2, mean2, rstd2 = flp.fused_layer_norm_forward(xs, w, center=center)
        dx2, _, _ = flp.fused_layer_norm_backward(_at(dy, lead, pad), xs, w, mean, rstd, center=center)
        assert torch.equal(rstd2, rstd) and (not center or torch.equal(mean2, mean))
        assert torch.equal(y2, y) and torch.equal(dx2, dx)
        flp.fused_layer_norm_forward(xs, w, center=center, y=xs)   # in place
        assert torch.equal(xs, y)
