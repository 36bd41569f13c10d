"""Ragged tiles of the 8-bit product's pairs, which leave C by boxes that two tiles in a row
share: with one or two K blocks a tile, an odd number of boxes in the last column of tiles and
several tiles a CTA pair, every element against the definition in 64 bits."""

import ctypes

import pytest
import torch

import selected_token_logprob_gb300 as flp
from selected_token_logprob_gb300 import _lib

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: U}
M, WHOLE = 38 * 256, 9 * 256   # with the ragged column 380 tiles of 256 x 256


def values(q, scale):
    s = scale.t().double().repeat_interleave(128, 1)[:, :q.shape[1]]
    if s.shape[0] != q.shape[0]:
        s = s.repeat_interleave(128, 0)[:q.shape[0]]
    return q.double() * s


# columns of the last tile: 1 or 3 boxes of one warp (64 columns of 16 bits, 32 of FP32), none of
# or one of the next's
@pytest.mark.parametrize("dtype,ragged", [(torch.bfloat16, 8), (torch.bfloat16, 64), (torch.float16, 136),
                                          (torch.bfloat16, 192), (torch.float32, 4), (torch.float32, 32),
                                          (torch.float32, 96), (torch.float32, 160)])
@pytest.mark.parametrize("square,k", [(True, 100), (True, 128), (False, 256)])
def test_ragged_tiles_in_a_row(square, k, dtype, ragged):
    n = WHOLE + ragged
    bn, split = ctypes.c_int(), ctypes.c_int()
    _lib.check("form", _lib.load().flp_selftest_fp8_form(M, n, k, square, 152, ctypes.byref(bn), ctypes.byref(split)))
    assert bn.value == 0   # the pairs
    g = torch.Generator(device="cuda").manual_seed(n + k)
    a = flp.quantize_fp8(torch.randn((M, k), generator=g, device="cuda"))
    b = flp.quantize_fp8(torch.randn((n, k), generator=g, device="cuda"), square)
    va, vb = values(a.q, a.scale), values(b.q, b.scale)
    want, size = va @ vb.t(), va.abs() @ vb.abs().t()
    # as the product's other tests: a block's 4 tensor-core steps lose 33 last places each of its sum of
    # magnitudes, the scales and the blocks' sums one rounding each; then half a step of the output
    tol = want.abs() * HALF[dtype] + 2.0 ** -24 + (135 + 2) * U * size * (1 + HALF[dtype])
    first = None
    for _ in range(4):
        c = flp.fp8_matmul(a.q, a.scale, b.q, b.scale, dtype)
        if first is None:
            first = c
            assert bool(((c.double() - want).abs() <= tol).all())
        assert torch.equal(c, first)
    assert flp.flp_device_error(0) == 0
