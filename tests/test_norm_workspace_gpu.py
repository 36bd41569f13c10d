"""GPU test: the norm's backward stays inside the scratch that its size function gives,
whatever the number of rows, and its results do not depend on a larger one."""

import pytest
import torch

import selected_token_logprob_gb300 as flp

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("n", [1, 2, 3, 17, 152, 305, 607, 1500])
@pytest.mark.parametrize("d", [4, 64, 250, 1031, 2048, 4096, 8192, 9001])
def test_exact_scratch(n, d):
    flp._lib.load(build_if_missing=True)
    g = torch.Generator(device=DEV).manual_seed(n + d)
    x = torch.randn(n, d, generator=g, device=DEV)
    dy = torch.randn(n, d, generator=g, device=DEV)
    _, mean, rstd = flp.fused_layer_norm_forward(x)
    need, most = flp.fused_layer_norm_backward_workspace_size(d, n), flp.fused_layer_norm_backward_workspace_size(d)
    assert need <= most
    buf = torch.full((need + 4096,), 171, dtype=torch.uint8, device=DEV)
    got = flp.fused_layer_norm_backward(dy, x, None, mean, rstd, workspace=buf[:need])
    assert (buf[need:] == 171).all()
    want = flp.fused_layer_norm_backward(dy, x, None, mean, rstd,
                                         workspace=torch.empty(most, dtype=torch.uint8, device=DEV))
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    xh = (x.double() - x.double().mean(1, keepdim=True)) / (x.double().var(1, keepdim=True, unbiased=False) + 1e-5).sqrt()
    if d > 4:   # an xh within 2^-15 of its size, and n sums: see test_norm_rows_gpu for the bound
        tol = (16 * (d / 32 + 64) + n + 64) * 2.0 ** -24 * 2 * (dy.double().abs() * (1 + xh.abs())).sum(0)
        assert ((got[1].double() - (dy.double() * xh).sum(0)).abs() <= tol).all()
    with pytest.raises(flp.FusedLogpError, match="workspace"):
        flp.fused_layer_norm_backward(dy, x, None, mean, rstd, workspace=buf[:need - 256])
