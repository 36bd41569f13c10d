"""8-bit products of CTA pairs into wider buffers: what lies behind C's last column stays, where that
column ends inside 16 bytes of a row that starts on such a boundary, too."""

import ctypes

import pytest
import torch

import selected_token_logprob_gb300 as flp
from selected_token_logprob_gb300 import _lib

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("m,n,k", [(939, 5523, 3002), (600, 1101, 520), (700, 1027, 700), (1025, 2049, 900), (513, 1150, 900)])
@pytest.mark.parametrize("square", [True, False])
def test_columns_behind(m, n, k, square, dtype):
    bn, split = ctypes.c_int(), ctypes.c_int()
    _lib.check("form", _lib.load().flp_selftest_fp8_form(m, n, k, square, 152, ctypes.byref(bn), ctypes.byref(split)))
    g = torch.Generator(device="cuda").manual_seed(n)
    a = flp.quantize_fp8(torch.randn((m, k), generator=g, device="cuda"))
    b = flp.quantize_fp8(torch.randn((n, k), generator=g, device="cuda"), square)
    want = flp.fp8_matmul(a.q, a.scale, b.q, b.scale, torch.float32).to(dtype)
    per = 16 // want.element_size()
    for more in (0, per, 5 * per):
        ld = -(-n // per) * per + more
        # the last row ends with its last column; what follows is not C's
        buf = torch.full((m * ld + 64,), 7.0, dtype=dtype, device="cuda")
        out = buf[:m * ld].view(m, ld)[:, :n]
        flp.fp8_matmul(a.q, a.scale, b.q, b.scale, out=out)
        assert torch.equal(out, want)
        out.fill_(7.0)
        assert bool((buf == 7.0).all())
    if m > 900:
        assert bn.value == 0   # the pairs
