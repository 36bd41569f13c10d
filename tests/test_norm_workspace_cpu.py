"""The scratch of the norm's backward: at most one partial row of dweight and one of
dbias a row of the batch."""

import ctypes

import pytest

from selected_token_logprob_gb300 import _lib
from selected_token_logprob_gb300 import build as flp_build


@pytest.fixture(scope="module")
def lib():
    flp_build.build()
    return _lib.load()


def _bytes(lib, d, n=None):
    b = ctypes.c_int64(-1)
    st = (lib.fused_layer_norm_backward_workspace_size(d, ctypes.byref(b)) if n is None else
          lib.fused_layer_norm_backward_rows_workspace_size(n, d, ctypes.byref(b)))
    return st, b.value


@pytest.mark.parametrize("d", [1, 64, 1031, 8192, 100000])
def test_few_rows_need_little(lib, d):
    row = 2 * 4 * ((d + 3) // 4 * 4)
    for n in (0, 1, 3, 100, 607):
        st, b = _bytes(lib, d, n)
        assert st == 0 and n * row <= b <= n * row + 256
    sizes = {_bytes(lib, d, n)[1] for n in (608, 609, 1 << 40)} | {_bytes(lib, d)[1]}
    assert len(sizes) == 1 and 607 * row < sizes.pop()


def test_refusals(lib):
    for d, n in ((0, 4), (-1, 4), (4, -1), (2 ** 62, 4), (2 ** 63 - 1, 1)):
        assert _bytes(lib, d, n)[0] == _lib.FLP_EINVAL
    assert lib.fused_layer_norm_backward_rows_workspace_size(4, 4, None) == _lib.FLP_EINVAL
