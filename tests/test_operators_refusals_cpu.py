"""Each refusal of the norm's, the preference loss's and the orthogonalised update's C
entries by its own message.  The unchanged arguments are host memory, which is refused
last, by the first CUDA call: a message that names the argument shows that its own check
spoke, and before that call."""

import ctypes

import pytest

from selected_token_logprob_gb300 import _lib
from selected_token_logprob_gb300 import build as flp_build
from test_operators_abi_cpu import BF16, F16, F32, _norm_bwd, _norm_fwd, _orth, _pref, _size

EINVAL, EUNSUP = _lib.FLP_EINVAL, _lib.FLP_EUNSUPPORTED
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    flp_build.build()
    return _lib.load()


@pytest.fixture(scope="module")
def p():
    buf = (ctypes.c_char * 65536)()
    p.keep = buf
    return (ctypes.addressof(buf) + 255) // 256 * 256


def _refused(lib, call, p, kw, status, *words):
    if callable(kw):
        kw = kw(p)
    assert call(lib, p, **kw) == status, kw
    text = lib.flp_last_error().decode()
    assert all(w in text for w in words), (kw, text)


def _late(lib, call, p):
    """The unchanged call is refused for its memory alone."""
    assert call(lib, p) == EINVAL
    text = lib.flp_last_error().decode()
    assert "cudaPointerGetAttributes" in text or "must point to device memory" in text, text


def test_norm_forward(lib, p):
    _late(lib, _norm_fwd, p)
    for kw, words in ((dict(n=-1), ("n must", "-1")), (dict(d=0), ("d must", "(got 0)")), (dict(dt=3), ("dtype", "got 3")),
                      (dict(dt=-1), ("dtype", "got -1")), (dict(wdt=F16), ("weight dtype", "got 1")),
                      (dict(ld=15), ("ld_x (15)",)), (dict(ld_y=15), ("ld_y (15)",)), (dict(eps=-1.0), ("eps", "-1")),
                      (dict(eps=NAN), ("eps", "nan")), (dict(eps=INF), ("eps", "inf")),
                      (dict(n=2 ** 62, ld=2 ** 20, ld_y=2 ** 20), ("extent overflows",)),
                      (dict(x=None), ("x is a null",)), (dict(y=None), ("y is a null",)),
                      (lambda p: dict(y=p + 8), ("y overlaps x",)), (lambda p: dict(y=p, ld_y=17), ("y overlaps x",)),
                      (lambda p: dict(y=p + 2 * (3 * 16 + 15)), ("y overlaps x",))):
        _refused(lib, _norm_fwd, p, kw, EINVAL, *words)
    _refused(lib, _norm_fwd, p, dict(d=2 ** 31, ld=2 ** 31, ld_y=2 ** 31), EUNSUP, "below 2^31")


def test_norm_backward(lib, p):
    _late(lib, _norm_bwd, p)
    for kw, words in ((dict(n=-1), ("n must", "-1")), (dict(d=0), ("d must",)), (dict(dt=3), ("dtype", "got 3")),
                      (dict(gdt=F16), ("dy dtype", "got 1")), (dict(wdt=F16), ("weight dtype", "got 1")),
                      (dict(ld=3), ("ld_x (3)",)), (dict(ld_dy=3), ("ld_dy (3)",)), (dict(ld_dx=3), ("ld_dx (3)",)),
                      (dict(wb=511), ("workspace_bytes (511)", "512")), (lambda p: dict(ws=p + 8), ("workspace", "16-byte")),
                      (lambda p: dict(dx=p + 2048), ("dx overlaps x",)), (lambda p: dict(dx=p), ("dx overlaps dy",)),
                      (lambda p: dict(dx=p + 16), ("dx overlaps dy",)),
                      (dict(n=2 ** 62, ld=2 ** 20, wb=2 ** 62), ("extent overflows",)),
                      (dict(rstd=None), ("rstd is a null",)), (dict(mean=None), ("mean is a null",)),
                      (dict(dx=None), ("dx is a null",)), (dict(ws=None), ("workspace is a null",))):
        _refused(lib, _norm_bwd, p, kw, EINVAL, *words)
    _refused(lib, _norm_bwd, p, dict(d=2 ** 31, ld=2 ** 31, ld_dy=2 ** 31, ld_dx=2 ** 31), EUNSUP, "below 2^31")
    assert _norm_bwd(lib, p, n=0, dw=None, db=None, wb=0, ws=None) == 0


def test_preference(lib, p):
    _late(lib, _pref, p)
    for kw, words in ((dict(n=-1), ("n must", "-1")), (dict(s=3), ("num_seqs", "got 3")), (dict(s=-2), ("num_seqs", "got -2")),
                      (dict(s=2 ** 31), ("num_seqs",)), (dict(kind=3), ("kind", "got 3")), (dict(kind=-1), ("kind", "got -1")),
                      (dict(layout=2), ("layout", "got 2")), (dict(beta=0.0), ("beta", "got 0")),
                      (dict(beta=-0.1), ("beta", "-0.1")), (dict(beta=NAN), ("beta", "nan")), (dict(beta=INF), ("beta", "inf")),
                      (dict(smooth=-0.1), ("label_smoothing", "-0.1")), (dict(smooth=1.5), ("label_smoothing", "1.5")),
                      (dict(smooth=NAN), ("label_smoothing", "nan")), (dict(kind=1, smooth=0.25), ("label_smoothing", "0.25")),
                      (dict(kind=2, smooth=0.25), ("label_smoothing",)), (dict(kind=2, margin=0.5), ("margin", "0.5")),
                      (dict(margin=INF), ("margin", "inf")), (dict(norm=-1.0), ("normalizer", "-1")),
                      (dict(norm=NAN), ("normalizer", "nan")), (dict(norm=INF), ("normalizer", "inf")),
                      (dict(wb=100), ("workspace_bytes (100)",)), (lambda p: dict(ws=p + 4), ("workspace", "16-byte")),
                      (dict(loss=None), ("loss is a null",)), (dict(logp=None), ("logp is a null",)),
                      (dict(grad=None), ("grad is a null",)), (dict(cu=None), ("cu_seqlens is a null",)),
                      (dict(rewards=None), ("rewards is a null",)), (dict(ws=None), ("workspace is a null",))):
        _refused(lib, _pref, p, kw, EINVAL, *words)


def test_orthogonalize(lib, p):
    _late(lib, _orth, p)
    for kw, words in ((dict(dt=5), ("dtype", "got 5")), (dict(odt=F16), ("out_dtype", "got 1")),
                      (dict(batch=-1), ("batch", "-1")), (dict(rows=-1), ("rows", "-1")), (dict(steps=0), ("steps", "got 0")),
                      (dict(steps=65), ("steps", "got 65")), (dict(coef=None), ("coefficients is a null",)),
                      (dict(coef=NAN), ("coefficients must be finite",)), (dict(coef=INF), ("coefficients must be finite",)),
                      (dict(eps=-1.0), ("eps",)), (dict(eps=INF), ("eps",)), (dict(eps=NAN), ("eps",)),
                      (dict(scale=NAN), ("scale",)), (dict(scale=INF), ("scale",)), (dict(ld=15), ("ld_x (15)",)),
                      (dict(ld_out=15), ("ld_out (15)",)),
                      (dict(batch=2, stride=-1, stride_out=128), ("stride_x must be >= 0",)),
                      (dict(batch=2, stride=128, stride_out=100), ("stride_out cover",)),
                      (dict(rows=4, ld=2 ** 62), ("extent overflows",)),
                      (dict(wb=100), ("workspace_bytes (100)",)), (lambda p: dict(ws=p + 16), ("workspace", "128-byte")),
                      (lambda p: dict(out=p + 64), ("out overlaps x",)),
                      (lambda p: dict(out=p, odt=BF16), ("out overlaps x",)),
                      (lambda p: dict(out=p, odt=F32, ld_out=24), ("out overlaps x",)),
                      (dict(x=None), ("x is a null",)), (dict(out=None), ("out is a null",))):
        _refused(lib, _orth, p, kw, EINVAL, *words)
    _refused(lib, _orth, p, dict(rows=70000, cols=70000, ld=70000, ld_out=70000), EUNSUP, "65536")


def test_sizes(lib):
    st, b = _size(lib, "logp_preference_loss_workspace_size", 2 ** 62, 2)
    assert st == 0 and 2 ** 62 // 512 * 8 < b < 2 ** 62 // 512 * 8 + 2 ** 20
    assert _size(lib, "logp_preference_loss_workspace_size", 2 ** 63 - 1, 2 ** 31 - 2)[0] == 0
    assert _size(lib, "fused_layer_norm_backward_workspace_size", 2 ** 60)[0] == EINVAL
    assert "overflows" in lib.flp_last_error().decode()
