"""GPU tests of the Newton-Schulz orthogonalisation against 64 bits.

Tolerance.  The kernels round four things: X's hi part and the off-diagonals of
A and B to FP16 (at a scale of 2^8), X's lo part to FP16 (2^11 finer), and the
output; the rest is FP32.  `_rounded` repeats those roundings on 64-bit
products, which gives the error E that the numerics cost for this very input.
The kernel's roundings are other draws of the same (its FP32 sums move some
values across a tie), so its distance to the exact result is at most 1.5 E +
2e-4 in the norm (for tiny matrices, where a handful of roundings do not
average, the constant covers them: one rounding is 2.4e-4 of a value), plus
the output type's own rounding, 2^-8 (BF16) at most.  E itself is below 3e-3
for these inputs; without the FP32 diagonals and lo it would reach 5e-2."""

import pytest
import torch

import selected_token_logprob_gb300 as flp

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ABC = flp.ORTHOGONALIZE_COEFFICIENTS


@pytest.fixture(scope="module", autouse=True)
def _built():
    flp._lib.load(build_if_missing=True)
    yield
    torch.cuda.synchronize()
    assert flp.flp_device_error(0) == 0


def _exact(x, coefs, eps=1e-7, scale=1.0):
    x = x.double()
    tall = x.shape[-2] > x.shape[-1]
    x = x.mT if tall else x
    x = x / (torch.linalg.vector_norm(x, dim=(-2, -1), keepdim=True) + eps)
    for a, b, c in coefs:
        q = x @ x.mT
        x = a * x + (b * q + c * (q @ q)) @ x
    return scale * (x.mT if tall else x)


def _rounded(x, coefs, eps=1e-7, scale=1.0):
    def h(v):
        return (v * 256).half().double() / 256

    x = x.double()
    tall = x.shape[-2] > x.shape[-1]
    x = x.mT if tall else x
    x = x / (torch.linalg.vector_norm(x, dim=(-2, -1), keepdim=True) + eps)
    for a, b, c in coefs:
        hi = h(x)
        x = hi + h((x - hi) * 2048) / 2048
        q = hi @ hi.mT
        d = q.diagonal(dim1=-2, dim2=-1)
        a0 = h(q - torch.diag_embed(d))
        sq = a0 @ a0
        p = (b + c * (d[..., :, None] + d[..., None, :])) * a0 + c * sq
        e = b * d + c * d * d + c * sq.diagonal(dim1=-2, dim2=-1)
        b0 = h(p - torch.diag_embed(p.diagonal(dim1=-2, dim2=-1)))
        x = (a + e)[..., None] * x + b0 @ hi
    return scale * (x.mT if tall else x)


def _rel(got, want):
    n = torch.linalg.vector_norm(want, dim=(-2, -1))
    return (torch.linalg.vector_norm(got.double() - want, dim=(-2, -1)) / n).max().item()


def _check(x, got, coefs, eps=1e-7, scale=1.0):
    want = _exact(x, coefs, eps, scale)
    tol = 1.5 * _rel(_rounded(x, coefs, eps, scale), want) + 2e-4 + (2.0 ** -8 if got.dtype == torch.bfloat16 else 0)
    err = _rel(got, want)
    assert got.shape == x.shape and err <= tol, (err, tol)
    return err


def _gradient(shape, seed, rank=None, floor=0.3, dtype=torch.float32):
    g = torch.Generator(device=DEV).manual_seed(seed)
    m, n = shape[-2:]
    r = rank or max(1, min(m, n) // 4)
    s = torch.arange(1, r + 1, device=DEV, dtype=torch.float32).pow(-0.5)
    x = (torch.randn(*shape[:-1], r, generator=g, device=DEV) * s) @ torch.randn(*shape[:-2], r, n, generator=g,
                                                                             device=DEV)
    return (1e-3 * (x + floor * torch.randn(*shape, generator=g, device=DEV))).to(dtype)


SHAPES = [(1, 1), (1, 17), (2, 3), (5, 5), (16, 4096), (31, 33), (33, 31), (63, 64), (64, 64), (65, 64), (64, 1024),
          (100, 1000), (127, 129), (128, 128), (129, 128), (130, 500), (192, 192), (200, 250), (256, 256),
          (257, 1023), (384, 640), (500, 70), (1001, 2050), (1024, 4096), (2050, 1001), (4097, 70), (2048, 2048),
          (8, 257), (70, 513), (128, 1025), (24, 2049), (2100, 127), (96, 4161), (128, 6144), (6100, 100), (20, 6145),
          (7000, 128)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_sizes(shape, out_dtype):
    x = _gradient(shape, shape[0] * 7 + shape[1])
    _check(x, flp.orthogonalize(x, out_dtype=out_dtype), [ABC] * 5)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("shape", [(3, 64, 96), (2, 130, 65), (5, 40, 200), (4, 256, 256), (2, 320, 1000),
                                   (3, 600, 300), (40, 100, 600), (20, 33, 4099), (12, 1500, 64)])
def test_stacks_and_types(dtype, shape):
    x = _gradient(shape, 3, dtype=dtype)
    got = flp.orthogonalize(x, out_dtype=torch.float32)
    _check(x, got, [ABC] * 5)
    assert torch.equal(got, flp.orthogonalize(x, out_dtype=torch.float32))
    for k in range(min(3, shape[0])):   # one alone (its sums may take another order)
        _check(x[k], flp.orthogonalize(x[k], out_dtype=torch.float32), [ABC] * 5)


@pytest.mark.parametrize("shape", [(26, 100, 4000), (26, 4100, 128), (40, 127, 2000), (30, 64, 1500), (9, 128, 520),
                                   (300, 24, 130), (14, 100, 900)])
def test_stacks_of_small_matrices(shape):
    """More matrices than clusters that run at once, and few enough for smaller slices."""
    x = _gradient(shape, 5)
    got = flp.orthogonalize(x, out_dtype=torch.float32)
    _check(x, got, [ABC] * 5)
    assert torch.equal(got, flp.orthogonalize(x, out_dtype=torch.float32))


@pytest.mark.parametrize("kind", ["gauss", "low_rank", "one_direction", "decaying", "orthogonal"])
@pytest.mark.parametrize("shape", [(256, 256), (512, 1500), (700, 128)])
def test_spectra(kind, shape):
    g = torch.Generator(device=DEV).manual_seed(8)
    m, n = shape
    if kind == "gauss":
        x = torch.randn(m, n, generator=g, device=DEV)
    elif kind == "low_rank":
        x = _gradient(shape, 9, rank=16, floor=1e-2)
    elif kind == "one_direction":
        x = torch.randn(m, 1, generator=g, device=DEV) @ torch.randn(1, n, generator=g, device=DEV)
    else:
        k = min(m, n)
        u = torch.linalg.qr(torch.randn(m, k, generator=g, device=DEV, dtype=torch.float64))[0]
        v = torch.linalg.qr(torch.randn(n, k, generator=g, device=DEV, dtype=torch.float64))[0]
        s = torch.arange(1, k + 1, device=DEV, dtype=torch.float64).pow(-1.0 if kind == "decaying" else 0.0)
        x = ((u * s) @ v.T).float()
    _check(x, flp.orthogonalize(x, out_dtype=torch.float32), [ABC] * 5)


def test_singular_values_come_near_one():
    x = _gradient((300, 900), 10, floor=1.0)
    s = torch.linalg.svdvals(flp.orthogonalize(x, out_dtype=torch.float32).double())
    assert s.min() > 0.5 and s.max() < 1.3


@pytest.mark.parametrize("steps", [1, 2, 3, 8])
def test_steps_schedules_scale_eps(steps):
    x = _gradient((150, 260), 11)
    _check(x, flp.orthogonalize(x, steps=steps, out_dtype=torch.float32, scale=-0.25), [ABC] * steps, scale=-0.25)
    coefs = [(2.0, -1.5 + 0.05 * k, 0.5) for k in range(steps)]
    _check(x, flp.orthogonalize(x, steps=steps, coefficients=coefs, eps=0.5, out_dtype=torch.float32), coefs, eps=0.5)


@pytest.mark.parametrize("pad,lead", [(0, 0), (1, 3), (8, 8), (24, 0)])
@pytest.mark.parametrize("shape", [(70, 130), (130, 70), (128, 256)])
def test_strides_and_alignment(shape, pad, lead):
    m, n = shape
    x = _gradient(shape, 12, dtype=torch.bfloat16)
    want = flp.orthogonalize(x)
    buf = torch.full((3 * m * (n + pad) + lead + 64,), float("nan"), device=DEV, dtype=torch.bfloat16)
    xin = torch.as_strided(buf, (3, m, n), (m * (n + pad), n + pad, 1), lead)
    xin[:] = x
    obuf = torch.full((3 * m * (n + pad + 2) + lead + 64,), 7.0, device=DEV, dtype=torch.bfloat16)
    out = torch.as_strided(obuf, (3, m, n), (m * (n + pad + 2), n + pad + 2, 1), lead)
    flp.orthogonalize(xin, out=out)
    for k in range(3):
        assert torch.equal(out[k], want)
    keep = torch.ones(obuf.numel(), dtype=torch.bool, device=DEV)
    torch.as_strided(keep, out.shape, out.stride(), lead).fill_(False)
    assert (obuf[keep] == 7.0).all()


def test_in_place_workspace_stream_and_graph():
    x = _gradient((200, 333), 13, dtype=torch.bfloat16)
    want = flp.orthogonalize(x)
    z = x.clone()
    assert flp.orthogonalize(z, out=z) is z and torch.equal(z, want)
    ws = torch.full((flp.orthogonalize_workspace_size(1, 200, 333),), 255, dtype=torch.uint8, device=DEV)
    assert torch.equal(flp.orthogonalize(x, workspace=ws), want)   # no initial contents are needed
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = flp.orthogonalize(x)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = flp.orthogonalize(x, workspace=ws)
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_zero_non_finite_and_empty():
    x = _gradient((3, 96, 160), 14)
    want = flp.orthogonalize(x)
    x[1] = 0
    got = flp.orthogonalize(x)
    assert torch.equal(got[0], want[0]) and (got[1] == 0).all() and torch.equal(got[2], want[2])
    for bad in (float("nan"), float("inf")):
        x[1, 5, 7] = bad
        got = flp.orthogonalize(x)
        assert torch.equal(got[0], want[0]) and got[1].isnan().all() and torch.equal(got[2], want[2])
    for shape in ((0, 5), (5, 0), (0, 4, 4), (2, 0, 3)):
        e = flp.orthogonalize(torch.empty(shape, device=DEV))
        assert e.shape == shape and e.dtype == torch.bfloat16


@pytest.mark.parametrize("magnitude", [1e-12, 1e-5, 1.0, 1e6, 1e15])
def test_magnitudes(magnitude):
    x = torch.randn(90, 300, device=DEV, generator=torch.Generator(device=DEV).manual_seed(15)) * magnitude
    _check(x, flp.orthogonalize(x, eps=0.0, out_dtype=torch.float32), [ABC] * 5, eps=0.0)


def test_refusals():
    x = torch.ones(8, 16, device=DEV)
    with pytest.raises(TypeError):
        flp.orthogonalize(x.double())
    with pytest.raises(TypeError):
        flp.orthogonalize(x, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        flp.orthogonalize(x.cpu())
    with pytest.raises(ValueError):
        flp.orthogonalize(x.t())
    with pytest.raises(ValueError):
        flp.orthogonalize(x[0])
    with pytest.raises(ValueError):
        flp.orthogonalize(x, steps=0)
    with pytest.raises(ValueError):
        flp.orthogonalize(x, coefficients=(1.0, 2.0))
    with pytest.raises(ValueError):
        flp.orthogonalize(x, coefficients=[(1.0, 2.0, 3.0)] * 4)
    with pytest.raises(ValueError):
        flp.orthogonalize(x, out=torch.empty(16, 8, device=DEV))
    for kw in (dict(steps=65), dict(eps=-1.0), dict(scale=float("inf")), dict(coefficients=(1.0, float("nan"), 0.0)),
               dict(workspace=torch.empty(64, dtype=torch.uint8, device=DEV))):
        with pytest.raises(flp.FusedLogpError):
            flp.orthogonalize(x, **kw)
    with pytest.raises(flp.FusedLogpError):   # shifted onto its own input
        buf = torch.ones(200, device=DEV)
        flp.orthogonalize(buf[:128].view(8, 16), out=buf[16:144].view(8, 16))
    with pytest.raises(flp.FusedLogpError):
        flp.orthogonalize_workspace_size(1, 70000, 70000)
