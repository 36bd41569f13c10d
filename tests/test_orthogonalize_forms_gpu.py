"""GPU tests of each form of the orthogonalised update's products against 64 bits: tiles
on clusters, persistent CTAs (128 x 128 tiles) and CTA pairs (256 x 256), for the
symmetric products and for those with X, at sides that end inside a tile and stacks
whose last tile reads into the next matrix.  The tolerance is test_orthogonalize_gpu's."""

import ctypes

import pytest
import torch

import selected_token_logprob_gb300 as flp
from test_orthogonalize_gpu import ABC, _check, _gradient

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
CLUSTER, CTA, PAIR = 0, 1, 2
#: shape, form of X X^T and A^2, form of the products with X (on 152 SMs, 76 pairs)
CASES = [((8, 1024, 1500), CTA, PAIR), ((8, 900, 1100), CTA, PAIR), ((13, 700, 900), CTA, PAIR),
         ((3000, 3100), CTA, PAIR), ((1, 3100, 3000), CTA, PAIR), ((6, 1100, 1200), CTA, PAIR),
         ((40, 300, 400), CTA, PAIR), ((100, 200, 130), CTA, PAIR), ((27, 310, 300), CTA, CTA),
         ((5, 1000, 1100), PAIR, PAIR), ((2, 2900, 2500), PAIR, PAIR), ((2, 2470, 2600), PAIR, PAIR),
         ((5, 1060, 1200), PAIR, PAIR), ((4096, 4096), PAIR, PAIR), ((3, 1700, 3333), PAIR, PAIR),
         ((1030, 5000), CLUSTER, PAIR), ((3, 600, 2000), CLUSTER, PAIR), ((20, 300, 310), CLUSTER, CTA),
         ((9, 600, 640), CLUSTER, CTA), ((257, 1023), CLUSTER, CLUSTER)]


@pytest.fixture(scope="module")
def lib():
    lib = flp._lib.load(build_if_missing=True)
    yield lib
    torch.cuda.synchronize()
    assert flp.flp_device_error(0) == 0


def _form(lib, product, shape):
    b, m, n = (1, *shape)[-3:]
    f = ctypes.c_int(-1)
    assert lib.flp_selftest_orthogonalize_form(product, b, m, n, 152, 76, ctypes.byref(f)) == 0
    return f.value


@pytest.mark.parametrize("shape,gram,apply", CASES)
def test_forms(lib, shape, gram, apply):
    assert (_form(lib, 0, shape), _form(lib, 1, shape)) == (gram, apply)
    x = _gradient(shape, 21)
    got = flp.orthogonalize(x, out_dtype=torch.float32)
    _check(x, got, [ABC] * 5)
    b, m, n = (1, *shape)[-3:]
    ws = torch.full((flp.orthogonalize_workspace_size(b, m, n),), 255, dtype=torch.uint8, device=DEV)
    assert torch.equal(flp.orthogonalize(x, out_dtype=torch.float32, workspace=ws), got)   # NaN everywhere before
    _check(x, flp.orthogonalize(x), [ABC] * 5)


@pytest.mark.parametrize("shape", [(8, 900, 1100), (13, 700, 900), (5, 1060, 1200), (2, 2470, 2600)])
def test_matrices_of_a_stack_stay_alone(lib, shape):
    x = _gradient(shape, 22)
    want = flp.orthogonalize(x, out_dtype=torch.float32)
    x[1] *= 2.0 ** 40
    x[0, 3, 5] = float("nan")
    got = flp.orthogonalize(x, out_dtype=torch.float32, eps=0.0)
    assert got[0].isnan().all() and got[1:].isfinite().all()
    x[0, 3, 5] = 0.0
    again = flp.orthogonalize(x, out_dtype=torch.float32, eps=0.0)
    assert torch.equal(again[1:], got[1:])
    _check(x[1], got[1], [ABC] * 5, eps=0.0)
    assert want[1:].isfinite().all()


def test_refusals(lib):
    f = ctypes.c_int(-1)
    for a in ((2, 1, 8, 8, 152, 76), (-1, 1, 8, 8, 152, 76), (0, -1, 8, 8, 152, 76), (0, 1, 8, 8, 0, 0)):
        assert lib.flp_selftest_orthogonalize_form(*a, ctypes.byref(f)) == flp._lib.FLP_EINVAL
    assert lib.flp_selftest_orthogonalize_form(0, 1, 8, 8, 152, 76, None) == flp._lib.FLP_EINVAL
