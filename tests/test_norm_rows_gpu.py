"""GPU tests of the norm's backward on grids wider than its rows need.

The CTAs that take rows are counted for 152 SMs and each writes one partial row of
dweight and dbias; more CTAs may be launched so that the partial rows are folded in one
turn.  `flp_selftest_norm_backward` sizes the rows' CTAs for fewer SMs, so that here,
too, CTAs are left over while the others take several rows each.

Tolerance of the sums, u = 2^-24: a row's xh is within 4 (d/32 + 64) u (1 + A) of its
size, A = mean|x| rstd, and the sum over n rows in any order within (n + 64) u, both of
sum |dy| (1 + |xh|).  dx does not depend on the grid: it has the public call's bits."""

import pytest
import torch

import selected_token_logprob_gb300 as flp

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24


@pytest.fixture(scope="module")
def lib():
    return flp._lib.load(build_if_missing=True)


def _backward(lib, sms, dy, x, w, mean, rstd, center):
    n, d = x.shape
    ws = torch.full((flp.fused_layer_norm_backward_workspace_size(d),), 255, dtype=torch.uint8, device=DEV)
    dx = torch.empty_like(x)
    dw, db = torch.empty(d, device=DEV), torch.empty(d, device=DEV)
    types = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
    st = lib.flp_selftest_norm_backward(
        sms, dy.data_ptr(), types[dy.dtype], dy.stride(0), x.data_ptr(), types[x.dtype], n, d, x.stride(0), w.data_ptr(),
        types[w.dtype], mean.data_ptr() if center else None, rstd.data_ptr(), 1 if center else 0, ws.data_ptr(),
        ws.numel(), dx.data_ptr(), d, dw.data_ptr(), db.data_ptr(), 0, torch.cuda.current_stream().cuda_stream)
    assert st == 0, lib.flp_last_error()
    return dx, dw, db


@pytest.mark.parametrize("d", [64, 120, 250, 512, 1031, 2048, 4096, 4500, 8192, 8191, 9001])
@pytest.mark.parametrize("n", [5, 700])
@pytest.mark.parametrize("sms", [1, 4])
@pytest.mark.parametrize("dtype,center", [(torch.bfloat16, True), (torch.float32, False)])
def test_sums_with_more_ctas_than_rows_take(lib, d, n, sms, dtype, center):
    g = torch.Generator(device=DEV).manual_seed(d + n)
    x = (torch.randn(n, d, generator=g, device=DEV) + 0.3).to(dtype)
    w = 1 + 0.2 * torch.randn(d, generator=g, device=DEV)
    dy = torch.randn(n, d, generator=g, device=DEV)
    _, mean, rstd = flp.fused_layer_norm_forward(x, w, center=center)
    want_dx, _, _ = flp.fused_layer_norm_backward(dy, x, w, mean, rstd, center=center)
    dx, dw, db = _backward(lib, sms, dy, x, w, mean, rstd, center)
    assert torch.equal(dx, want_dx)
    x64, dy64 = x.double(), dy.double()
    mu = x64.mean(1, keepdim=True) if center else 0.0
    rs = 1 / ((x64 - mu).square().mean(1, keepdim=True) + 1e-5).sqrt()
    xh = (x64 - mu) * rs
    a = (x64.abs().mean(1, keepdim=True) * rs).max()
    tol = (16 * (d / 32 + 64) + n + 64) * U * (1 + a) * (dy64.abs() * (1 + xh.abs())).sum(0)
    assert ((dw.double() - (dy64 * xh).sum(0)).abs() <= tol).all()
    assert ((db.double() - dy64.sum(0)).abs() <= tol).all()
    again = _backward(lib, sms, dy, x, w, mean, rstd, center)
    assert torch.equal(again[1], dw) and torch.equal(again[2], db)


def test_refusals(lib):
    for sms in (0, -1, 153):
        a = [sms, None, 2, 8, None, 2, 1, 8, 8, None, 2, None, None, 0, None, 0, None, 8, None, None, 0, None]
        assert lib.flp_selftest_norm_backward(*a) == flp._lib.FLP_EINVAL and b"sms" in lib.flp_last_error()
