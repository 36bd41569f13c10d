"""GPU tests of the orthogonalised update over the whole range of finite inputs.

A power of two takes no rounding, so with eps = 0 the update of 2^k x has the bits of the
update of x, whatever k, while no value of 2^k x leaves the normal numbers: that is
exact, for every type and for values whose squares FP32 cannot hold.  The update of
x itself is held to 64 bits by test_orthogonalize_gpu, whose check the large matrices
here take, too."""

import pytest
import torch

import selected_token_logprob_gb300 as flp
from test_orthogonalize_gpu import _check

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
#: One CTA, a cluster of several, tall and unaligned; tiles on clusters and persistent.
SHAPES = [(30, 100), (100, 1000), (70, 513), (2100, 127), (200, 250), (257, 1023), (1001, 600), (3, 300, 700),
          (2, 128, 640), (1500, 2600)]


@pytest.fixture(scope="module", autouse=True)
def _built():
    flp._lib.load(build_if_missing=True)
    yield
    torch.cuda.synchronize()
    assert flp.flp_device_error(0) == 0


def _matrix(shape, seed, dtype=torch.float32):
    """Values between 2^-8 and 2^2 in size, or 0: times 2^k they stay normal numbers."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(shape, generator=g, device=DEV).clamp(-3.9, 3.9)
    return torch.where(x.abs() < 2.0 ** -8, torch.zeros_like(x), x).to(dtype)


def _ortho(x, eps=0.0):
    return flp.orthogonalize(x, eps=eps, out_dtype=torch.float32)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_powers_of_two_change_no_bit(shape, dtype):
    x = _matrix(shape, 1, dtype)
    want = _ortho(x)
    assert want.isfinite().all() and want.abs().max() > 0
    for k in (-118, -90, -62, -41, 31, 49, 56, 63, 64, 90, 125):
        assert torch.equal(_ortho(x * 2.0 ** k), want), k


def test_fp16_values_of_every_size():
    x = _matrix((90, 300), 2, torch.float16)
    want = _ortho(x)
    for k in (-6, 13):
        assert torch.equal(_ortho(x * 2.0 ** k), want), k


@pytest.mark.parametrize("shape", [(100, 1000), (513, 700)])
def test_one_large_part_and_matrices_of_unlike_sizes(shape):
    """Rows so unlike that their sums of squares need scales of their own: what is far
    below the largest does not count, and no matrix of a stack takes another's scale."""
    x = _matrix((3, *shape), 3)
    want = _ortho(x)
    sizes = torch.tensor([2.0 ** 100, 1.0, 2.0 ** -100], device=DEV)[:, None, None]
    assert torch.equal(_ortho(x * sizes), want)
    y = x[0] * 2.0 ** -100
    y[7] = x[0, 7] * 2.0 ** 100
    z = torch.zeros_like(y)
    z[7] = x[0, 7]
    assert torch.equal(_ortho(y), _ortho(z))


@pytest.mark.parametrize("shape", [(64, 64), (100, 1000), (300, 400), (2, 40, 50)])
def test_zeros_and_eps(shape):
    for dtype in (torch.float32, torch.bfloat16):
        z = torch.zeros(shape, device=DEV, dtype=dtype)
        for eps in (0.0, 1e-40, 1e-7):
            assert (_ortho(z, eps) == 0).all(), eps
    # eps counts at its own size, however the squares are scaled: |x| = 2^k, eps = 2^k, so X has the norm 1/2
    x = torch.zeros(shape, device=DEV)
    x[..., 3, 5] = 1.0
    coefs = [(1.0, 0.0, 0.0)]
    for k in (-100, -3, 80):
        got = flp.orthogonalize(x * 2.0 ** k, steps=1, coefficients=coefs, eps=2.0 ** k, out_dtype=torch.float32)
        assert torch.equal(got, x / 2), k


@pytest.mark.parametrize("magnitude", [1e17, 3e37, 1e-30])
def test_large_matrices_at_the_ends_of_the_range(magnitude):
    x = torch.randn(1024, 4096, device=DEV, generator=torch.Generator(device=DEV).manual_seed(4)).clamp(-4, 4) * magnitude
    _check(x, _ortho(x), [flp.ORTHOGONALIZE_COEFFICIENTS] * 5, eps=0.0)


@pytest.mark.parametrize("shape", [(3, 60, 100), (3, 300, 200)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_non_finite_matrices_stay_alone(shape, bad):
    x = _matrix(shape, 5) * 2.0 ** 100
    want = _ortho(x)
    x[1, 5, 7] = bad
    got = _ortho(x)
    assert torch.equal(got[0], want[0]) and got[1].isnan().all() and torch.equal(got[2], want[2])
