"""The 8-bit product's waits end: by the abort flag of their CTA at once, by the clock alone in a
few seconds, which is reported in the device error word."""

import ctypes
import time

import pytest
import torch

import selected_token_logprob_gb300 as flp
from selected_token_logprob_gb300 import _lib

pytestmark = pytest.mark.gpu


def waited(aborted):
    out = ctypes.c_int(-1)
    torch.cuda.synchronize()
    t0 = time.monotonic()
    _lib.check("wait", _lib.load().flp_selftest_fp8_wait(0, aborted, ctypes.byref(out)))
    assert out.value == 1
    return time.monotonic() - t0


def test_an_abort_ends_every_wait():
    waited(1)                    # the first launch loads the kernel
    assert waited(1) < 0.25
    assert flp.flp_device_error(0) == 0


def test_the_clock_ends_the_wait():
    """A tick of the clock's upper half: 2^32 cycles, 2.1 s at 2070 MHz; at least 1000 are assumed."""
    assert waited(0) < 4.5
    assert flp.flp_device_error(0) == 1
    assert flp.flp_device_error(0) == 0
    x = flp.quantize_fp8(torch.ones((4, 128), device="cuda"))
    assert bool((flp.fp8_matmul(x.q, x.scale, x.q, x.scale) == 128).all())
    assert flp.flp_device_error(0) == 0
