"""The refusal of the self-test of the 8-bit product's waits, on the host."""

from selected_token_logprob_gb300 import _lib
from selected_token_logprob_gb300 import build as flp_build


def test_refusal():
    flp_build.build()
    lib = _lib.load()
    assert lib.flp_selftest_fp8_wait(0, 1, None) == _lib.FLP_EINVAL
    assert "gave_up" in lib.flp_last_error().decode()
