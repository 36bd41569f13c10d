"""GPU tests of the preference loss against plain formulas in 64 bits.

Tolerances, u = 2^-24.  A sequence's sum over 512-token chunks rounds each
difference once and adds at most 2 + 4 + 5 times in FP32 (the rest is a sum of two
floats), so its log-ratio is within e_s = 16 u sum|logp - ref| (/ n_s when averaging) and
h within e = e_c + e_j.  u = beta h - margin is rounded once.
  rewards |err| <= beta e_s + u |reward|
  pair    sigmoid, hinge: beta e + 8 u (1 + |u| + l); ipo: (2 |t| + e) e + 4 u l
  loss    the mean of the pairs' bounds, + 2 u |loss|
  dl/dh   sigmoid: beta (beta e + 8 u (1 + |u|)) (the logistic is 1/4-Lipschitz and
          exp(u) magnifies the rounding of u by |u|); ipo: 2 e + 4 u |t|; hinge:
          exact away from the kink
  grad    that / D (/ n_s), + 8 u |grad|"""

import math

import numpy as np
import pytest
import torch

import selected_token_logprob_gb300 as flp

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    flp._lib.load(build_if_missing=True)


def _plain(logp, ref, mask, cu, kind, beta, smooth, margin, average, layout, normalizer):
    """(loss, grad, rewards) and their tolerances, in 64 bits."""
    n, seqs = len(logp), len(cu) - 1
    d = logp if ref is None else logp - ref
    r, cnt, err = np.zeros(seqs), np.zeros(seqs, dtype=int), np.zeros(seqs)
    for s in range(seqs):
        at = np.arange(cu[s], cu[s + 1])
        at = at[mask[at]]
        cnt[s] = len(at)
        r[s] = d[at].sum()
        err[s] = 16 * U * np.abs(d[at]).sum()
        if average and len(at):
            r[s] /= len(at)
            err[s] /= len(at)
    half = seqs // 2
    pairs = [(p, p + half) if layout == "halves" else (2 * p, 2 * p + 1) for p in range(half)]
    live = [p for p, (c, j) in enumerate(pairs) if cnt[c] and cnt[j]]
    den = normalizer if normalizer > 0 else len(live)
    loss = loss_tol = 0.0
    grad, gtol = np.zeros(n), np.zeros(n)
    for p in live:
        c, j = pairs[p]
        h, e = r[c] - r[j], err[c] + err[j]
        u = beta * h - margin
        if kind == "sigmoid":
            l = (1 - smooth) * np.logaddexp(0, -u) + smooth * np.logaddexp(0, u)
            # both terms by themselves: their sum smooth - 1 + sigma(u) cancels for a large u
            dh = beta * (smooth * math.exp(-np.logaddexp(0, -u)) - (1 - smooth) * math.exp(-np.logaddexp(0, u)))
            lt, dt = beta * e + 8 * U * (1 + abs(u) + l), beta * (beta * e + 8 * U * (1 + abs(u)))
        elif kind == "hinge":
            l, dh = max(0.0, 1 - u), (-beta if u < 1 else 0.0)
            lt, dt = beta * e + 8 * U * (1 + abs(u) + l), 0.0
            assert abs(u - 1) > 1e-4
        else:
            t = h - 0.5 / beta
            l, dh = t * t, 2 * t
            lt, dt = (2 * abs(t) + e) * e + 4 * U * l, 2 * e + 4 * U * abs(t)
        loss += l
        loss_tol += lt
        for s, sign in ((c, 1), (j, -1)):
            at = np.arange(cu[s], cu[s + 1])
            at = at[mask[at]]
            w = 1 / len(at) if average else 1.0
            grad[at] = sign * dh * w / den
            gtol[at] = dt * w / den + 8 * U * np.abs(grad[at])
    if live:
        loss, loss_tol = loss / den, loss_tol / den + 2 * U * abs(loss / den)
    rewards = np.array([[beta * r[c], beta * r[j]] for c, j in pairs]).reshape(half, 2)
    rtol = np.array([[beta * err[c], beta * err[j]] for c, j in pairs]).reshape(half, 2) + U * np.abs(rewards)
    return loss, grad, rewards, loss_tol, gtol, rtol


def _case(lens, seed, masked=0.3, lead=0, tail=0, junk=True, ref=True):
    g = torch.Generator().manual_seed(seed)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64) + lead
    n = int(cu[-1]) + tail
    logp = -torch.rand(n, generator=g).double() ** 3 * 8
    logp = logp.float()
    r = (logp + 0.3 * torch.randn(n, generator=g)).float() if ref else None
    mask = torch.rand(n, generator=g) >= masked
    if junk:
        at = ~mask & (torch.rand(n, generator=g) < 0.5)
        logp = torch.where(at, torch.tensor(float("-inf")), logp)
        if ref:
            r = torch.where(at, torch.tensor(float("nan")), r)
    return logp, r, mask, cu


def _both(logp, ref, mask, cu, **kw):
    kw = dict(kind="sigmoid", beta=0.1, label_smoothing=0.0, margin=0.0, average=False, layout="interleaved",
              normalizer=0.0) | kw
    got = flp.logp_preference_loss(logp.to(DEV), torch.from_numpy(cu).to(DEV),
                                   ref_logp=None if ref is None else ref.to(DEV),
                                   active_mask=None if mask is None else mask.to(DEV), **kw)
    m = np.ones(len(logp), dtype=bool) if mask is None else mask.numpy()
    clean = np.where(m, logp.double().numpy(), 0.0)
    cref = None if ref is None else np.where(m, ref.double().numpy(), 0.0)
    want = _plain(clean, cref, m, cu, kw["kind"], kw["beta"], kw["label_smoothing"], kw["margin"], kw["average"],
                  kw["layout"], kw["normalizer"])
    return [t.double().cpu().numpy() for t in got], want


def _check(got, want):
    loss, grad, rewards = got
    wl, wg, wr, tl, tg, tr = want
    assert abs(loss[0] - wl) <= tl + 1e-30, (loss[0], wl, tl)
    assert np.all(np.abs(grad - wg) <= tg + 1e-38), np.max(np.abs(grad - wg) - tg)
    assert np.all(np.abs(rewards - wr) <= tr + 1e-38)
    assert np.all(grad[wg == 0] == 0)


LENS = {
    "ones": [1] * 6,
    "pair": [5, 9],
    "tile_edges": [256, 256, 255, 257, 512, 1, 1, 511, 128, 384],
    "empties": [0, 4, 7, 0, 0, 0, 300, 20, 0, 0],
    "long": [70000, 3, 9, 33333],
    "ragged": [int(v) for v in torch.randint(0, 900, (400,), generator=torch.Generator().manual_seed(4))],
    "short": [int(v) for v in torch.randint(0, 9, (3000,), generator=torch.Generator().manual_seed(5))],
    "none": [],
    "all_empty": [0, 0, 0, 0],
}


@pytest.mark.parametrize("lens", sorted(LENS))
@pytest.mark.parametrize("kind", ["sigmoid", "hinge", "ipo"])
@pytest.mark.parametrize("layout", ["interleaved", "halves"])
def test_kinds_and_layouts(lens, kind, layout):
    logp, ref, mask, cu = _case(LENS[lens], 11)
    _check(*_both(logp, ref, mask, cu, kind=kind, layout=layout))


@pytest.mark.parametrize("smooth,margin", [(0.0, 0.0), (0.1, 0.0), (0.5, 0.7), (1.0, -2.0)])
@pytest.mark.parametrize("average,ref", [(True, False), (True, True), (False, False)])
def test_smoothing_margin_average_reference(smooth, margin, average, ref):
    logp, r, mask, cu = _case(LENS["ragged"], 12, ref=ref)
    _check(*_both(logp, r, mask, cu, beta=2.0 if average else 0.05, label_smoothing=smooth, margin=margin,
                  average=average))


@pytest.mark.parametrize("lead,tail", [(0, 0), (1, 0), (300, 700), (0, 1)])
def test_tokens_outside_and_normalizer(lead, tail):
    logp, ref, mask, cu = _case(LENS["tile_edges"], 13, lead=lead, tail=tail)
    got, want = _both(logp, ref, mask, cu, normalizer=37.0)
    _check(got, want)
    assert np.all(got[1][:lead] == 0) and np.all(got[1][len(logp) - tail:] == 0)
    _check(*_both(logp, ref, None if torch.isfinite(logp).all() else mask, cu))


def test_no_mask_and_all_masked():
    logp, ref, mask, cu = _case(LENS["ragged"], 14, junk=False)
    _check(*_both(logp, ref, None, cu))
    got, want = _both(logp, ref, torch.zeros_like(mask), cu)
    _check(got, want)
    assert got[0][0] == 0 and np.all(got[1] == 0) and np.all(got[2] == 0)
    got, _ = _both(logp, ref, torch.zeros_like(mask), cu, normalizer=4.0)
    assert got[0][0] == 0 and np.all(got[1] == 0)


@pytest.mark.parametrize("shift", [1, 2, 3])
def test_unaligned_arrays_give_the_same_bits(shift):
    logp, ref, mask, cu = _case(LENS["ragged"], 15)
    n = len(logp)

    def moved(t):
        b = torch.empty(n + 8, dtype=t.dtype, device=DEV)
        b[shift:shift + n] = t.to(DEV)
        return b[shift:shift + n]

    c = torch.from_numpy(cu).to(DEV)
    a = flp.logp_preference_loss(logp.to(DEV), c, ref_logp=ref.to(DEV), active_mask=mask.to(DEV))
    b = flp.logp_preference_loss(moved(logp), c, ref_logp=moved(ref), active_mask=moved(mask))
    for x, y in zip(a, b):
        assert torch.equal(x, y)


def test_non_finite_tokens_stay_in_their_pair():
    logp, ref, mask, cu = _case([300, 280, 500, 10, 40, 60], 16, masked=0.0)
    clean = _both(logp, ref, mask, cu)[0]
    bad = logp.clone()
    bad[cu[2] + 5] = float("nan")
    got = _both(bad, ref, mask, cu)[0]
    assert math.isnan(got[0][0]) and np.isnan(got[2][1, 0]) and np.isfinite(got[2][1, 1])
    assert np.isnan(got[1][cu[2]:cu[4]]).all()
    assert np.array_equal(got[1][:cu[2]], clean[1][:cu[2]]) and np.array_equal(got[1][cu[4]:], clean[1][cu[4]:])
    # an impossible rejected answer: its pair is won, without NaN
    bad = logp.clone()
    bad[cu[3]] = float("-inf")
    got = _both(bad, ref, mask, cu)[0]
    assert math.isfinite(got[0][0]) and np.isfinite(got[1]).all() and np.all(got[1][cu[2]:cu[4]] == 0)
    assert got[2][1, 1] == -math.inf
    # and an impossible chosen one: infinite loss, finite gradient
    bad = logp.clone()
    bad[cu[2]] = float("-inf")
    got = _both(bad, ref, mask, cu)[0]
    assert got[0][0] == math.inf and np.isfinite(got[1]).all()


def test_extreme_margins():
    lens = [4, 4] * 3
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
    logp = torch.zeros(24)
    for p, h in enumerate((300.0, -300.0, 0.0)):
        logp[8 * p] = h
    for kind in ("sigmoid", "hinge", "ipo"):
        _check(*_both(logp, None, None, cu, kind=kind, beta=1.0))


def test_gradient_against_differences():
    """Central differences of the 64-bit loss, step 1e-4: their error is
    O(1e-8 beta^3); the kernel's grad is FP32."""
    logp, ref, mask, cu = _case([7, 5, 12, 3], 17)
    for kw in (dict(beta=0.7, label_smoothing=0.2, margin=0.3), dict(kind="ipo", beta=0.5),
               dict(kind="hinge", beta=0.01), dict(beta=1.5, average=True)):
        got, _ = _both(logp, ref, mask, cu, **kw)
        full = dict(kind="sigmoid", beta=0.1, label_smoothing=0.0, margin=0.0, average=False, layout="interleaved",
                    normalizer=0.0) | kw
        m = mask.numpy()
        x = np.where(m, logp.double().numpy(), 0.0)
        r = np.where(m, ref.double().numpy(), 0.0)
        for t in range(len(x)):
            hi, lo = x.copy(), x.copy()
            hi[t] += 1e-4
            lo[t] -= 1e-4
            f = [_plain(v, r, m, cu, full["kind"], full["beta"], full["label_smoothing"], full["margin"],
                        full["average"], full["layout"], 0.0)[0] for v in (hi, lo)]
            num = (f[0] - f[1]) / 2e-4 if m[t] else 0.0
            assert abs(got[1][t] - num) <= 1e-6 * max(1.0, np.max(np.abs(got[1]))) + 1e-7


def test_repeats_streams_and_graph():
    logp, ref, mask, cu = _case(LENS["ragged"], 18)
    d = [logp.to(DEV), torch.from_numpy(cu).to(DEV), ref.to(DEV), mask.to(DEV)]
    ws = torch.empty(flp.logp_preference_loss_workspace_size(len(logp), len(cu) - 1), dtype=torch.uint8, device=DEV)

    def call():
        return flp.logp_preference_loss(d[0], d[1], ref_logp=d[2], active_mask=d[3], workspace=ws)

    ws.fill_(255)   # no initial contents are needed
    want = call()
    for _ in range(3):
        for x, y in zip(want, call()):
            assert torch.equal(x, y)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = call()
    torch.cuda.current_stream().wait_stream(side)
    for x, y in zip(want, got):
        assert torch.equal(x, y)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = call()
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    for x, y in zip(want, got):
        assert torch.equal(x, y)


def test_batch_larger_than_one_wave():
    """2^24 + 321 tokens: every CTA of both token passes takes several chunks."""
    n = 2 ** 24 + 321
    g = torch.Generator(device=DEV).manual_seed(1)
    logp = -torch.rand(n, generator=g, device=DEV)
    ref = logp + 0.1 * torch.randn(n, generator=g, device=DEV)
    cuts = torch.sort(torch.randint(0, n + 1, (4095,), generator=g, device=DEV)).values
    cu = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), cuts, torch.full((1,), n, device=DEV)])
    loss, grad, rewards = flp.logp_preference_loss(logp, cu, ref_logp=ref, kind="ipo", beta=0.1)
    d = torch.cat([torch.zeros(1, dtype=torch.float64, device=DEV), (logp.double() - ref.double()).cumsum(0)])
    r = d[cu[1:]] - d[cu[:-1]]
    lens = cu.diff()
    h = r[0::2] - r[1::2]
    live = (lens[0::2] > 0) & (lens[1::2] > 0)
    t = torch.where(live, h - 5.0, 0.0)
    want = (t * t).sum() / live.sum()
    assert abs(loss.double()[0] - want) <= 1e-4 * want
    assert (rewards.double() - 0.1 * torch.stack([r[0::2], r[1::2]], 1)).abs().max() <= 1e-4
    dr = torch.stack([2 * t, -2 * t], 1).reshape(-1) / live.sum()
    assert (grad.double() - torch.repeat_interleave(dr, lens)).abs().max() <= 1e-4 * dr.abs().max()


def test_tokens_without_sequences():
    """No sequences: cu_seqlens and rewards may be null at the C entry."""
    n = 1500
    logp, grad, loss = torch.zeros(n, device=DEV), torch.full((n,), 7.0, device=DEV), torch.full((1,), 7.0, device=DEV)
    size = flp.logp_preference_loss_workspace_size(n, 0)
    ws = torch.empty(size, dtype=torch.uint8, device=DEV)
    st = flp._lib.load().logp_preference_loss(logp.data_ptr(), None, None, None, 0, n, 0, 0, 0, 0.1, 0.0, 0.0, 0.0,
                                              ws.data_ptr(), size, loss.data_ptr(), grad.data_ptr(), None,
                                              torch.cuda.current_stream().cuda_stream)
    assert st == 0
    assert float(loss) == 0 and torch.count_nonzero(grad) == 0


@pytest.mark.parametrize("mean", [1, 3, 9, 31, 40, 70])
def test_many_short_sequences(mean):
    rng = np.random.default_rng(mean)
    lens = [int(v) for v in rng.integers(0, 2 * mean + 1, 700)] + [2000, 5, 0, 33]
    logp, ref, mask, cu = _case(lens, 40 + mean)
    _check(*_both(logp, ref, mask, cu))
    logp, ref, _, cu = _case(lens, 50 + mean, junk=False)
    _check(*_both(logp, ref, None, cu, average=True, kind="ipo", layout="halves"))


def test_one_sequence_of_more_than_2_31_tokens():
    """Token offsets and a sequence's count past 32 bits.  The chosen answer's
    logp is -2^-10 everywhere and the rejected one's -2^-9 (exact in every
    partial sum up to the chunks'), so h = 2^-10 up to the mean's rounding."""
    long, short = (1 << 31) + 777, 1000
    n = long + short
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB of free device memory")
    logp = torch.full((n,), -2.0 ** -10, device=DEV)
    logp[long:] = -2.0 ** -9
    cu = torch.tensor([0, long, n], device=DEV)
    loss, grad, rewards = flp.logp_preference_loss(logp, cu, beta=0.5, average=True)
    u = 0.5 * 2.0 ** -10
    dh = -0.5 / (1 + math.exp(u))
    assert abs(float(loss) - math.log1p(math.exp(-u))) < 1e-6
    assert rewards[0].tolist() == pytest.approx([-u, -2 * u], rel=1e-6)
    at = torch.tensor([0, 12345, (1 << 31) - 1, 1 << 31, long - 1], device=DEV)
    assert grad[at].tolist() == pytest.approx([dh / long] * 5, rel=1e-6)
    assert grad[long:].tolist() == pytest.approx([-dh / short] * short, rel=1e-6)
    del logp, grad
    torch.cuda.empty_cache()


def test_refusals():
    logp, ref, mask, cu = _case([5, 9], 19)
    d, c = logp.to(DEV), torch.from_numpy(cu).to(DEV)
    for kw in (dict(kind="dpo"), dict(layout="rows")):
        with pytest.raises(ValueError):
            flp.logp_preference_loss(d, c, **kw)
    for kw in (dict(beta=0.0), dict(beta=float("inf")), dict(label_smoothing=1.5),
               dict(kind="ipo", label_smoothing=0.1), dict(kind="ipo", margin=1.0), dict(margin=float("nan")),
               dict(normalizer=-1.0), dict(workspace=torch.zeros(16, dtype=torch.uint8, device=DEV))):
        with pytest.raises(flp.FusedLogpError):
            flp.logp_preference_loss(d, c, **kw)
    with pytest.raises(ValueError):
        flp.logp_preference_loss(d, c[:2])      # one sequence
    with pytest.raises(ValueError):
        flp.logp_preference_loss(d, c.int())
    with pytest.raises(TypeError):
        flp.logp_preference_loss(d.half(), c)
    with pytest.raises(ValueError):
        flp.logp_preference_loss(d, c, ref_logp=ref[:3].to(DEV))
    with pytest.raises(ValueError):
        flp.logp_preference_loss(logp, c)
