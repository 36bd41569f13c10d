"""GPU tests of the norm in front of the LM head (layer norm, RMS norm) against
plain formulas in 64 bits.

Tolerances.  u = 2^-24 (FP32), h = half an ulp of the output's type relative
to the value (2^-9 BF16, 2^-12 FP16 times 2 for the binade, u FP32).  A sum of
k FP32 terms in any fixed order of at most d/32 + 32 serial steps is within
G = (d/32 + 64) u of its terms' absolute sum.  With A = mean|x| rstd (how much
larger the row's values are than its spread: the mean's error is G mean|x|):
  y      |err| <= h |y| + 4 G (1 + A) (|w| (1 + |xh|) + |b|)
  dx     |err| <= h |dx| + 4 G (1 + A) rstd (|g| + mean|g| + |xh| mean|g xh| + mean|g|)
  dw, db |err| <= (4 G + (n/32 + 64) u) (1 + max A) sum_rows |dy| (1 + |xh|)"""

import pytest
import torch

import selected_token_logprob_gb300 as flp

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
HALF_ULP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: U}


@pytest.fixture(scope="module", autouse=True)
def _built():
    flp._lib.load(build_if_missing=True)


def _rows(n, d, dtype, gen, pad=0, lead=0, offset=0.0, scale=1.0):
    """[n, d] rows inside a wider buffer, `lead` elements after its start."""
    buf = torch.full((n * (d + pad) + lead + 8,), float("nan"), dtype=dtype, device=DEV)
    v = buf[lead:lead + n * (d + pad)].view(n, d + pad)[:, :d]
    v.copy_(torch.randn((n, d), generator=gen, device=DEV) * scale + offset)
    return v


def _reference(x, w, b, eps, center, dy=None):
    x = x.double()
    w = torch.ones(x.shape[1], device=DEV, dtype=torch.float64) if w is None else w.double()
    b = torch.zeros_like(w) if b is None else b.double()
    mu = x.mean(1, keepdim=True) if center else torch.zeros_like(x[:, :1])
    rstd = 1 / ((x - mu).square().mean(1, keepdim=True) + eps).sqrt()
    xh = (x - mu) * rstd
    out = {"mu": mu, "rstd": rstd, "xh": xh, "y": xh * w + b, "A": x.abs().mean(1, keepdim=True) * rstd}
    if dy is not None:
        dy = dy.double()
        g = dy * w
        t = g - xh * (g * xh).mean(1, keepdim=True) - (g.mean(1, keepdim=True) if center else 0)
        out |= {"g": g, "dx": t * rstd, "dw": (dy * xh).sum(0), "db": dy.sum(0)}
    return out


def _check(x, w, b, eps, center, dy, got):
    y, mean, rstd, dx, dw, db = got
    n, d = x.shape
    r = _reference(x, w, b, eps, center, dy)
    G = (d / 32 + 64) * U
    h = HALF_ULP[x.dtype]
    aw = 1.0 if w is None else w.double().abs()
    ab = 0.0 if b is None else b.double().abs()
    tol = h * r["y"].abs() + 4 * G * (1 + r["A"]) * (aw * (1 + r["xh"].abs()) + ab) + 1e-30
    if x.dtype == torch.float16:
        tol = tol + 2.0 ** -25   # half a step of the subnormals
    assert ((y.double() - r["y"]).abs() <= tol).all()
    if center:
        assert ((mean.double() - r["mu"][:, 0]).abs() <= G * x.double().abs().mean(1) + 1e-30).all()
    else:
        assert mean is None
    assert ((rstd.double() / r["rstd"][:, 0] - 1).abs() <= 4 * G * (1 + r["A"][:, 0]) ** 2 + 4 * U).all()
    if dy is None:
        return
    ag = r["g"].abs().mean(1, keepdim=True)
    agx = (r["g"] * r["xh"]).abs().mean(1, keepdim=True)
    tol = (h * r["dx"].abs() + 4 * G * (1 + r["A"]) * r["rstd"] * (r["g"].abs() + 2 * ag + r["xh"].abs() * agx)
           + 1e-30)
    if x.dtype == torch.float16:
        tol = tol + 2.0 ** -25
    assert ((dx.double() - r["dx"]).abs() <= tol).all()
    gn = (4 * G + (n / 32 + 64) * U) * (1 + r["A"].max())
    ady = dy.double().abs()
    if dw is not None:
        assert ((dw.double() - r["dw"]).abs() <= gn * (ady * (1 + r["xh"].abs())).sum(0) + 1e-30).all()
    if db is not None:
        assert ((db.double() - r["db"]).abs() <= gn * ady.sum(0) + 1e-30).all()


def _run(x, w, b, eps, center, dy):
    y, mean, rstd = flp.fused_layer_norm_forward(x, w, b, eps=eps, center=center)
    dx, dw, db = flp.fused_layer_norm_backward(dy, x, w, mean, rstd, center=center, with_dweight=w is not None,
                                               with_dbias=b is not None)
    return y, mean, rstd, dx, dw, db


SHAPES = [(1, 1), (3, 2), (2, 7), (5, 31), (4, 32), (1, 33), (9, 64), (17, 100), (2, 255), (300, 256), (33, 257),
          (6, 520), (305, 1000), (12, 1024), (11, 1031), (4, 2048), (7, 2056), (3, 4095), (613, 4096), (5, 5000),
          (3, 8192), (2, 8200), (2, 16384), (3, 16390), (2, 40000)]


@pytest.mark.parametrize("n,d", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("center", [True, False])
def test_forward_and_backward(n, d, dtype, center):
    gen = torch.Generator(device=DEV).manual_seed(n * 65537 + d)
    x = _rows(n, d, dtype, gen, offset=0.3)
    w = (1 + 0.3 * torch.randn(d, generator=gen, device=DEV)).to(dtype)
    b = (0.3 * torch.randn(d, generator=gen, device=DEV)).to(dtype) if center else None
    dy = _rows(n, d, dtype, gen)
    _check(x, w, b, 1e-5, center, dy, _run(x, w, b, 1e-5, center, dy))


@pytest.mark.parametrize("n,d", [(1000, 128), (1001, 65), (30011, 64), (40000, 100), (6007, 16), (20003, 129), (9001, 256),
                                 (2050, 200), (77, 513), (5003, 768), (6001, 1024), (4001, 1001)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("center", [True, False])
def test_many_narrow_rows(n, d, dtype, center):
    """Rows that share a warp or a CTA, more of them than run at once."""
    gen = torch.Generator(device=DEV).manual_seed(n * 65537 + d)
    x = _rows(n, d, dtype, gen, offset=0.3)
    w = (1 + 0.3 * torch.randn(d, generator=gen, device=DEV)).to(dtype)
    b = (0.3 * torch.randn(d, generator=gen, device=DEV)).to(dtype) if center else None
    dy = _rows(n, d, dtype, gen)
    got = _run(x, w, b, 1e-5, center, dy)
    _check(x, w, b, 1e-5, center, dy, got)
    for p, q in zip(got, _run(x, w, b, 1e-5, center, dy)):
        assert p is None and q is None or torch.equal(p, q)


@pytest.mark.parametrize("d", [64, 250, 1024, 1031, 4096])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("wide_dy,wide_w", [(True, True), (True, False), (False, True)])
def test_mixed_types(d, dtype, wide_dy, wide_w):
    gen = torch.Generator(device=DEV).manual_seed(d)
    n = 77
    x = _rows(n, d, dtype, gen)
    wdt = torch.float32 if wide_w else dtype
    w = (1 + 0.3 * torch.randn(d, generator=gen, device=DEV)).to(wdt)
    b = (0.3 * torch.randn(d, generator=gen, device=DEV)).to(wdt)
    dy = _rows(n, d, torch.float32 if wide_dy else dtype, gen)
    for center in (True, False):
        _check(x, w, b, 1e-6, center, dy, _run(x, w, b, 1e-6, center, dy))


@pytest.mark.parametrize("d", [96, 1000, 1024, 4096])
@pytest.mark.parametrize("pad,lead", [(8, 0), (1, 0), (0, 1), (5, 3), (64, 4)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strides_and_alignment(d, pad, lead, dtype):
    """Rows of wider buffers at any element offset; what lies between the rows
    is NaN and must not be touched."""
    gen = torch.Generator(device=DEV).manual_seed(d + pad)
    n = 41
    x = _rows(n, d, dtype, gen, pad, lead)
    dy = _rows(n, d, dtype, gen, pad=lead, lead=pad)
    wbuf = torch.randn(d + 3, generator=gen, device=DEV).to(dtype)
    w, b = wbuf[lead % 3:lead % 3 + d], wbuf[3 - lead % 3:3 - lead % 3 + d]
    y, dx = _rows(n, d, dtype, gen, pad, lead), _rows(n, d, dtype, gen, pad=pad + 2, lead=lead)
    y, mean, rstd = flp.fused_layer_norm_forward(x, w, b, y=y)
    dx, dw, db = flp.fused_layer_norm_backward(dy, x, w, mean, rstd, dx=dx)
    _check(x, w, b, 1e-5, True, dy, (y, mean, rstd, dx, dw, db))
    for t, p, at in ((y, pad, lead), (dx, pad + 2, lead)):
        whole = t._base
        keep = torch.ones(whole.numel(), dtype=torch.bool, device=DEV)
        torch.as_strided(keep, t.shape, t.stride(), at).fill_(False)
        assert whole[keep].isnan().all()


@pytest.mark.parametrize("d", [128, 1031, 4096])
def test_rows_are_independent_of_the_batch(d):
    gen = torch.Generator(device=DEV).manual_seed(5)
    x, dy = _rows(700, d, torch.bfloat16, gen), _rows(700, d, torch.bfloat16, gen)
    w = torch.randn(d, generator=gen, device=DEV).bfloat16()
    a = _run(x, w, None, 1e-5, True, dy)
    for k in (0, 333, 699):
        o = _run(x[k:k + 1], w, None, 1e-5, True, dy[k:k + 1])
        for p, q in zip(a[:4], o[:4]):
            assert torch.equal(p[k:k + 1], q)
    again = _run(x, w, None, 1e-5, True, dy)
    for p, q in zip(a[:5], again[:5]):
        assert torch.equal(p, q)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [72, 1024, 2049])
def test_extreme_rows(dtype, d):
    """A constant row (no spread), a zero row, a row far from zero, a row of
    huge and of tiny values; a row with an infinity or NaN spoils only itself."""
    gen = torch.Generator(device=DEV).manual_seed(d)
    x = _rows(9, d, dtype, gen)
    x[0] = 0.0
    x[1] = 3.0
    x[2] = x[2] + 200.0
    x[3] *= 1e15
    x[4] *= 1e-15
    dy = _rows(9, d, dtype, gen)
    w = torch.ones(d, device=DEV, dtype=dtype)
    for center in (True, False):
        _check(x[:7], w, None, 1e-5, center, dy[:7], _run(x[:7], w, None, 1e-5, center, dy[:7]))
    clean = _run(x, w, None, 1e-5, True, dy)
    bad = x.clone()
    bad[7, d // 2] = float("inf")
    bad[8, 0] = float("nan")
    y, _, _, dx, dw, _ = _run(bad, w, None, 1e-5, True, dy)
    assert torch.equal(y[:7], clean[0][:7]) and torch.equal(dx[:7], clean[3][:7])
    assert not y[7].isfinite().any() and y[8].isnan().all() and dx[8].isnan().all() and dw.isnan().all()


def test_in_place_no_vectors_and_other_stream():
    gen = torch.Generator(device=DEV).manual_seed(1)
    x = _rows(33, 512, torch.float16, gen)
    want, mean, rstd = flp.fused_layer_norm_forward(x)
    _check(x, None, None, 1e-5, True, None, (want, mean, rstd, None, None, None))
    z = x.clone()
    flp.fused_layer_norm_forward(z, y=z)
    assert torch.equal(z, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = flp.fused_layer_norm_forward(x)[0]
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)


@pytest.mark.parametrize("d", [520, 1024, 4096])
def test_accumulate_and_empty(d):
    gen = torch.Generator(device=DEV).manual_seed(3)
    x, dy = _rows(50, d, torch.bfloat16, gen), _rows(50, d, torch.bfloat16, gen)
    w = torch.randn(d, generator=gen, device=DEV).bfloat16()
    _, mean, rstd = flp.fused_layer_norm_forward(x, w)
    _, dw, db = flp.fused_layer_norm_backward(dy, x, w, mean, rstd)
    aw, ab = torch.full_like(dw, 2.0), torch.full_like(db, -1.0)
    flp.fused_layer_norm_backward(dy, x, w, mean, rstd, dweight=aw, dbias=ab, accumulate=True)
    assert torch.equal(aw, 2.0 + dw) and torch.equal(ab, -1.0 + db)
    e = x[:0]
    y, m, r = flp.fused_layer_norm_forward(e, w)
    assert y.shape == (0, d) and m.shape == (0,)
    dx, zw, zb = flp.fused_layer_norm_backward(dy[:0], e, w, m, r)
    assert dx.shape == (0, d) and (zw == 0).all() and (zb == 0).all()
    flp.fused_layer_norm_backward(dy[:0], e, w, m, r, dweight=aw, dbias=ab, accumulate=True)
    assert torch.equal(aw, 2.0 + dw)


@pytest.mark.parametrize("center", [True, False])
@pytest.mark.parametrize("d", [40, 1024])
def test_gradient_against_differences(center, d):
    """<dx, v> against central differences of sum(dy y) in 64 bits along v:
    their error is O(t^2) (about 1e-8 here), the kernel's that of FP32."""
    gen = torch.Generator(device=DEV).manual_seed(d)
    n, t = 6, 1e-4
    x, dy = _rows(n, d, torch.float32, gen), _rows(n, d, torch.float32, gen)
    w = torch.randn(d, generator=gen, device=DEV)
    b = torch.randn(d, generator=gen, device=DEV)
    got = _run(x, w, b, 1e-5, center, dy)

    def f(x_, w_, b_):
        return (dy.double() * _reference(x_, w_, b_, 1e-5, center)["y"]).sum()

    v = torch.randn(n, d, generator=gen, device=DEV).double()
    u = torch.randn(d, generator=gen, device=DEV).double()
    X, W, B = x.double(), w.double(), b.double()
    for grad, along, hi, lo in ((got[3], v, (X + t * v, W, B), (X - t * v, W, B)),
                                (got[4], u, (X, W + t * u, B), (X, W - t * u, B)),
                                (got[5], u, (X, W, B + t * u), (X, W, B - t * u))):
        num = (f(*hi) - f(*lo)) / (2 * t)
        scale = (grad.double().abs() * along.abs()).sum()
        assert abs((grad.double() * along).sum() - num) <= 2e-5 * scale


def test_autograd():
    gen = torch.Generator(device=DEV).manual_seed(9)
    x = _rows(20, 256, torch.float32, gen).clone().requires_grad_()
    w = torch.randn(256, generator=gen, device=DEV).requires_grad_()
    b = torch.randn(256, generator=gen, device=DEV).requires_grad_()
    y = flp.fused_layer_norm(x, w, b)
    y.sum().backward()   # a broadcast upstream gradient
    dy = torch.ones_like(y)
    r = _run(x.detach(), w.detach(), b.detach(), 1e-5, True, dy)
    assert torch.equal(x.grad, r[3]) and torch.equal(w.grad, r[4]) and torch.equal(b.grad, r[5])
    z = flp.fused_layer_norm(x.detach().bfloat16(), w, center=False)
    z.float().square().sum().backward()
    assert w.grad.isfinite().all()


def test_graph_replay():
    gen = torch.Generator(device=DEV).manual_seed(2)
    x, dy = _rows(64, 1024, torch.bfloat16, gen), _rows(64, 1024, torch.bfloat16, gen)
    w = torch.randn(1024, generator=gen, device=DEV).bfloat16()
    want = _run(x, w, None, 1e-5, True, dy)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = _run(x, w, None, 1e-5, True, dy)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    for p, q in zip(want[:5], got[:5]):
        assert torch.equal(p, q)


def test_refusals():
    x = torch.zeros(4, 16, device=DEV)
    w = torch.ones(16, device=DEV)
    with pytest.raises(TypeError):
        flp.fused_layer_norm_forward(x.double())
    with pytest.raises(TypeError):
        flp.fused_layer_norm_forward(x, w.half())
    with pytest.raises(ValueError):
        flp.fused_layer_norm_forward(x, w[:15])
    with pytest.raises(ValueError):
        flp.fused_layer_norm_forward(x, w.cpu())
    with pytest.raises(ValueError):
        flp.fused_layer_norm_forward(x, w, eps=float("nan"))
    with pytest.raises(ValueError):
        flp.fused_layer_norm_forward(x.t())
    with pytest.raises(flp.FusedLogpError):   # shifted onto its own input
        buf = torch.zeros(100, device=DEV)
        flp.fused_layer_norm_forward(buf[:64].view(4, 16), y=buf[8:72].view(4, 16))
    y, m, r = flp.fused_layer_norm_forward(x, w)
    with pytest.raises(ValueError):
        flp.fused_layer_norm_backward(x, x, w, None, r)
    with pytest.raises(ValueError):
        flp.fused_layer_norm_backward(x[:3], x, w, m, r)
    with pytest.raises(ValueError):
        flp.fused_layer_norm_backward(x, x, w, m, r, accumulate=True)
    with pytest.raises(flp.FusedLogpError):
        flp.fused_layer_norm_backward(x, x, w, m, r, dx=x)
    with pytest.raises(flp.FusedLogpError):
        flp.fused_layer_norm_backward(x, x, w, m, r, workspace=torch.zeros(16, dtype=torch.uint8, device=DEV))
