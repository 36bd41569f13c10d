"""GPU tests of the orthogonalised update's accuracy against 64 bits, over spectra from
alike to rank 1 and over numbers of steps.

The kernels round X's hi part, and the off-diagonals of A and B, to FP16, and X's lo part
2^11 finer; lo takes a row of B by its diagonal f alone, where that is not noise, and in
the one-cluster form all of B but for the last steps (`_rounded`, which repeats those
roundings on 64-bit products).  The sums are FP32: a product adds up to 8 times into an
accumulator, each time cutting off at most 2^-23 of it, and the steps to come multiply
that noise by a each where a singular value is near zero.  So each case is within
  1.5 times the error of `_rounded` on this very input + 2e-4 (other draws of the same
  roundings, as in test_orthogonalize_gpu) + 2^-20 a^(steps - 1),
and within the ceiling that the header states for the usual coefficients: `_rounded` is
off by at most 3.5e-3 (5 steps), 3.9e-3 (6), 7.1e-3 (8) and 1.7e-2 (10) of the result's
norm over such spectra, and 2^-20 a^(steps - 1) is 1.3e-4, 4.6e-4, 5.5e-3 and 6.5e-2."""

import pytest
import torch

import selected_token_logprob_gb300 as flp
from test_orthogonalize_gpu import ABC, _exact, _rel

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
CEILING = {1: 1e-3, 2: 1e-3, 3: 4e-3, 5: 4e-3, 6: 4.5e-3, 8: 1.5e-2, 10: 8e-2}


@pytest.fixture(scope="module", autouse=True)
def _built():
    flp._lib.load(build_if_missing=True)
    yield
    torch.cuda.synchronize()
    assert flp.flp_device_error(0) == 0


def _rounded(x, coefs, eps=1e-7):
    def h(v):
        return (v * 256).half().double() / 256

    x = x.double()
    tall = x.shape[-2] > x.shape[-1]
    x = x.mT if tall else x
    one_cluster = x.shape[0] <= 128 and x.shape[1] <= 6144
    x = x / (torch.linalg.vector_norm(x) + eps)
    for k, (a, b, c) in enumerate(coefs):
        grow = 1.0
        for later in coefs[k + 1:]:
            grow *= later[0] ** 2
        hi = h(x)
        lo = x - hi if one_cluster else h((x - hi) * 2048) / 2048
        q = hi @ hi.mT
        d = q.diagonal()
        a0 = h(q - torch.diag(d))
        sq = a0 @ a0
        p = (b + c * (d[:, None] + d[None, :])) * a0 + c * sq
        e = b * d + c * d * d + c * sq.diagonal()
        keeps = sq.diagonal() <= 35.0 / grow * (d * d + sq.diagonal())
        f = e if one_cluster else torch.where(keeps, e, 0.0)
        b0 = h(p - torch.diag(p.diagonal()))
        takes = hi + h(lo) if one_cluster and grow > 35 else hi
        x = (a + e)[:, None] * hi + (a + f)[:, None] * lo + b0 @ takes
    return x.mT if tall else x


def _bound(x, coefs, want):
    return 1.5 * _rel(_rounded(x, coefs), want) + 2e-4 + 2.0 ** -20 * coefs[0][0] ** (len(coefs) - 1)


def _spectrum(kind, shape, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device=DEV)   # noqa: E731
    m, n = shape
    k = min(shape)
    name, _, arg = kind.partition(" ")
    if name == "gauss":
        return rand(m, n)
    if name == "rank":          # of exactly this share of the smaller side
        r = max(1, int(float(arg) * k))
        return rand(m, r) @ rand(r, n)
    if name == "floor":         # rank 4 over a floor
        s = torch.arange(1, 5, device=DEV).pow(-0.5)
        return 1e-3 * ((rand(m, 4) * s) @ rand(4, n) + float(arg) * rand(m, n))
    if name == "one":           # one direction, `arg` of it in a single row of the smaller side
        u = rand(k, 1)
        u[0] = 0
        u *= (1 - float(arg)) ** 0.5 / torch.linalg.vector_norm(u)
        u[0] = float(arg) ** 0.5
        x = u @ rand(1, max(shape)) + 1e-4 * rand(k, max(shape))
        return x if m <= n else x.T.contiguous()
    u = torch.linalg.qr(rand(m, k).double())[0]
    v = torch.linalg.qr(rand(n, k).double())[0]
    s = torch.ones(k, device=DEV, dtype=torch.float64)
    s[int(float(arg) * k):] = 0   # alike, and zero beyond
    return ((u * s) @ v.T).float()


KINDS = ["gauss", "alike 1", "alike 0.9", "rank 0.01", "rank 0.5", "rank 0.7", "rank 0.9", "floor 0.3", "floor 1e-2",
         "floor 1e-3", "floor 1e-5", "one 0.5", "one 0.8", "one 0.9", "one 0.97"]


@pytest.mark.parametrize("shape", [(8, 40), (60, 64), (128, 700), (1024, 100), (256, 256), (512, 2048), (700, 130)])
@pytest.mark.parametrize("kind", KINDS)
def test_spectra_and_steps(kind, shape):
    x = _spectrum(kind, shape, 31)
    for steps, ceiling in CEILING.items():
        coefs = [ABC] * steps
        want = _exact(x, coefs)
        err = _rel(flp.orthogonalize(x, steps=steps, out_dtype=torch.float32), want)
        if kind in ("alike 1", "floor 0.3"):   # no singular value near zero
            ceiling = min(ceiling, 4e-3)
        assert err <= min(_bound(x, coefs, want), ceiling), (steps, err)


@pytest.mark.parametrize("kind", ["gauss", "rank 0.5", "floor 1e-3"])
@pytest.mark.parametrize("shape", [(1100, 3000), (2600, 2700)])
def test_large(kind, shape):
    x = _spectrum(kind, shape, 32)
    for steps in (5, 8):
        coefs = [ABC] * steps
        want = _exact(x, coefs)
        err = _rel(flp.orthogonalize(x, steps=steps, out_dtype=torch.float32), want)
        assert err <= min(_bound(x, coefs, want), CEILING[steps]), (steps, err)


def test_coefficients_that_converge():
    """These bring every singular value to 1 and keep it there, and no noise is left to be
    multiplied: many steps are as accurate as a few."""
    for a, b, c, steps in ((2.0, -1.5, 0.5, 12), (1.5, -0.5, 0.0, 16), (15 / 8, -10 / 8, 3 / 8, 20)):
        for shape in ((100, 300), (300, 400)):
            x = _spectrum("floor 0.3", shape, 33)
            coefs = [(a, b, c)] * steps
            want = _exact(x, coefs)
            err = _rel(flp.orthogonalize(x, steps=steps, coefficients=coefs, out_dtype=torch.float32), want)
            assert err <= 1.5 * _rel(_rounded(x, coefs), want) + 2e-4 + 2.0 ** -20, (a, shape, err)


@pytest.mark.parametrize("m,n", [(2, 2), (2, 5), (5, 3), (4, 9), (7, 7), (8, 8), (40, 8), (16, 16), (32, 32), (64, 80)])
@pytest.mark.parametrize("kind", ["gauss", "rank 1", "rank 1 over 1e-3", "half rank", "rows of unlike size"])
def test_many_small_matrices(m, n, kind):
    """The header's ceilings on every matrix of a stack of hundreds."""
    g = torch.Generator(device=DEV).manual_seed(35)
    rand = lambda *s: torch.randn(500, *s, generator=g, device=DEV)   # noqa: E731
    r = max(1, min(m, n) // 2)
    x = {"gauss": lambda: rand(m, n), "rank 1": lambda: rand(m, 1) @ rand(1, n),
         "rank 1 over 1e-3": lambda: rand(m, 1) @ rand(1, n) + 1e-3 * rand(m, n),
         "half rank": lambda: rand(m, r) @ rand(r, n),
         "rows of unlike size": lambda: rand(m, n) * torch.exp(2 * rand(m, 1))}[kind]()
    tiny = min(m, n) < 8
    for steps, ceiling in ((5, 1e-2 if tiny else 4e-3), (8, 3e-2 if tiny else 1.5e-2)):
        want = _exact(x, [ABC] * steps)
        assert _rel(flp.orthogonalize(x, steps=steps, out_dtype=torch.float32), want) <= ceiling, steps


def test_a_stack_decides_row_by_row():
    """Matrices of unlike spectra in one stack keep their own bits."""
    x = torch.stack([_spectrum(k, (300, 500), 34) for k in ("gauss", "rank 0.01", "rank 0.5")])
    got = flp.orthogonalize(x, out_dtype=torch.float32)
    for k in range(3):
        want = _exact(x[k], [ABC] * 5)
        assert _rel(got[k], want) <= _bound(x[k], [ABC] * 5, want)
