"""Host-side checks of the norm's, the preference loss's and the orthogonalised
update's C entries: every refusal here is made before the first CUDA call."""

import ctypes

import pytest

from selected_token_logprob_gb300 import _lib
from selected_token_logprob_gb300 import build as flp_build

EINVAL, EUNSUP = _lib.FLP_EINVAL, _lib.FLP_EUNSUPPORTED
BF16, F16, F32 = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    flp_build.build()
    return _lib.load()


@pytest.fixture(scope="module")
def p():
    buf = (ctypes.c_char * 65536)()
    p.keep = buf
    return (ctypes.addressof(buf) + 255) // 256 * 256


def _size(lib, fn, *args):
    b = ctypes.c_int64(-1)
    return getattr(lib, fn)(*args, ctypes.byref(b)), b.value


def test_workspace_sizes(lib):
    st, small = _size(lib, "fused_layer_norm_backward_workspace_size", 8)
    st2, large = _size(lib, "fused_layer_norm_backward_workspace_size", 4096)
    assert st == st2 == 0 and 0 < small < large and large % 256 == 0
    assert _size(lib, "fused_layer_norm_backward_workspace_size", 0)[0] == EINVAL
    assert _size(lib, "fused_layer_norm_backward_workspace_size", 2 ** 60)[0] == EINVAL
    st, a = _size(lib, "logp_preference_loss_workspace_size", 0, 0)
    st2, b = _size(lib, "logp_preference_loss_workspace_size", 2 ** 24, 16384)
    assert st == st2 == 0 and 0 < a < b < 2 ** 21 * 4
    for n, s in ((-1, 0), (10, 3), (10, -2), (10, 2 ** 31)):
        assert _size(lib, "logp_preference_loss_workspace_size", n, s)[0] == EINVAL
    assert _size(lib, "logp_preference_loss_workspace_size", 2 ** 62, 2)[0] in (0, EINVAL)
    st, a = _size(lib, "flp_orthogonalize_workspace_size", 1, 64, 64)
    st2, b = _size(lib, "flp_orthogonalize_workspace_size", 2, 64, 100)
    assert st == st2 == 0 and 0 < a < b
    assert _size(lib, "flp_orthogonalize_workspace_size", -1, 4, 4)[0] == EINVAL
    for shape in ((1, 70000, 70000), (1, 2 ** 31, 4), (2 ** 30, 64, 64), (2 ** 24, 4096, 4096)):
        assert _size(lib, "flp_orthogonalize_workspace_size", *shape)[0] == EUNSUP
    for fn in ("fused_layer_norm_backward_workspace_size", "logp_preference_loss_workspace_size",
               "flp_orthogonalize_workspace_size"):
        n = len(_lib.SIGNATURES[fn][1]) - 1
        assert getattr(lib, fn)(*([4] * n), None) == EINVAL


def _norm_fwd(lib, p, **kw):
    a = dict(x=p, dt=BF16, n=4, d=16, ld=16, w=p, b=None, wdt=BF16, eps=1e-5, center=1, y=p + 4096, ld_y=16, mean=p,
             rstd=p) | kw
    return lib.fused_layer_norm_forward(a["x"], a["dt"], a["n"], a["d"], a["ld"], a["w"], a["b"], a["wdt"], a["eps"],
                                        a["center"], a["y"], a["ld_y"], a["mean"], a["rstd"], None)


def test_norm_forward_refusals(lib, p):
    for kw in (dict(n=-1), dict(d=0), dict(dt=3), dict(wdt=F16), dict(ld=15), dict(ld_y=15), dict(eps=-1.0),
               dict(eps=float("nan")), dict(n=2 ** 62, ld=2 ** 20, ld_y=2 ** 20), dict(y=p + 8), dict(x=None), dict(y=None),
               dict()):   # the last: host memory
        assert _norm_fwd(lib, p, **kw) == EINVAL, kw
        assert lib.flp_last_error()
    assert _norm_fwd(lib, p, d=2 ** 31, ld=2 ** 31, ld_y=2 ** 31) == EUNSUP
    assert _norm_fwd(lib, p, n=0, x=None, y=None) == 0


def _norm_bwd(lib, p, **kw):
    a = dict(dy=p, gdt=F32, ld_dy=16, x=p + 2048, dt=BF16, n=4, d=16, ld=16, w=p, wdt=F32, mean=p, rstd=p, center=1,
             ws=p + 8192, wb=2 ** 20, dx=p + 4096, ld_dx=16, dw=p, db=p, acc=0) | kw
    return lib.fused_layer_norm_backward(a["dy"], a["gdt"], a["ld_dy"], a["x"], a["dt"], a["n"], a["d"], a["ld"], a["w"],
                                         a["wdt"], a["mean"], a["rstd"], a["center"], a["ws"], a["wb"], a["dx"],
                                         a["ld_dx"], a["dw"], a["db"], a["acc"], None)


def test_norm_backward_refusals(lib, p):
    for kw in (dict(gdt=F16), dict(ld_dy=3), dict(ld_dx=3), dict(wb=16), dict(ws=p + 8), dict(dx=p + 2048),
               dict(dx=p + 16), dict(mean=None), dict(rstd=None), dict()):
        assert _norm_bwd(lib, p, **kw) == EINVAL, kw
    assert _norm_bwd(lib, p, n=0, dw=None, db=None) == 0


def _pref(lib, p, **kw):
    a = dict(logp=p, ref=None, mask=None, cu=p, s=2, n=10, kind=0, layout=0, avg=0, beta=0.1, smooth=0.0, margin=0.0,
             norm=0.0, ws=p, wb=2 ** 20, loss=p, grad=p, rewards=p) | kw
    return lib.logp_preference_loss(a["logp"], a["ref"], a["mask"], a["cu"], a["s"], a["n"], a["kind"], a["layout"],
                                    a["avg"], a["beta"], a["smooth"], a["margin"], a["norm"], a["ws"], a["wb"],
                                    a["loss"], a["grad"], a["rewards"], None)


def test_preference_refusals(lib, p):
    nan, inf = float("nan"), float("inf")
    for kw in (dict(n=-1), dict(s=3), dict(s=-2), dict(kind=3), dict(kind=-1), dict(layout=2), dict(beta=0.0),
               dict(beta=nan), dict(beta=inf), dict(smooth=-0.1), dict(smooth=1.1), dict(smooth=nan),
               dict(kind=1, smooth=0.1), dict(kind=2, margin=0.5), dict(margin=inf), dict(norm=-1.0), dict(norm=nan),
               dict(wb=100), dict(ws=p + 4), dict(logp=None), dict(cu=None), dict(loss=None), dict()):
        assert _pref(lib, p, **kw) == EINVAL, kw
        assert lib.flp_last_error()


def _orth(lib, p, **kw):
    a = dict(x=p, dt=F32, batch=1, rows=8, cols=16, ld=16, stride=0, steps=5, coef=True, eps=1e-7, scale=1.0, ws=p,
             wb=2 ** 24, out=p + 8192, odt=BF16, ld_out=16, stride_out=0) | kw
    c = (ctypes.c_float * 192)(*([1.0] * 192))
    if a["coef"] is not True and a["coef"] is not None:
        c[4] = a["coef"]
    return lib.flp_orthogonalize(a["x"], a["dt"], a["batch"], a["rows"], a["cols"], a["ld"], a["stride"], a["steps"],
                                 None if a["coef"] is None else c, a["eps"], a["scale"], a["ws"], a["wb"], a["out"],
                                 a["odt"], a["ld_out"], a["stride_out"], None)


def test_orthogonalize_refusals(lib, p):
    nan, inf = float("nan"), float("inf")
    for kw in (dict(dt=5), dict(odt=F16), dict(batch=-1), dict(rows=-1), dict(steps=0), dict(steps=65), dict(coef=None),
               dict(coef=nan), dict(eps=-1.0), dict(eps=inf), dict(scale=nan), dict(ld=15), dict(ld_out=15),
               dict(batch=2, stride=-1, stride_out=128), dict(batch=2, stride=128, stride_out=100), dict(wb=100),
               dict(ws=p + 16), dict(out=p + 64), dict(out=p, odt=BF16), dict(x=None), dict(out=None), dict()):
        assert _orth(lib, p, **kw) == EINVAL, kw
        assert lib.flp_last_error()
    assert _orth(lib, p, rows=70000, cols=70000, ld=70000, ld_out=70000) == EUNSUP
    for kw in (dict(batch=0), dict(rows=0), dict(cols=0, ld=0, ld_out=0)):
        assert _orth(lib, p, **kw) == 0
