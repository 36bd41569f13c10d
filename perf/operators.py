"""Operators of one preference-tuning step around the selected-token logp,
as measured cases: the norm in front of the LM head (layer norm or, without
centring, RMS norm; forward and backward with the weight's gradient), the
preference loss on packed pairs of sequences (loss, token gradients, rewards)
and the Newton-Schulz orthogonalisation of a weight's update.

Every case runs either in a plain form (elementary torch operations in FP32,
rounded once at the end) or, with ``own`` set, through this package's calls.
"""

import math

import torch

own = False

#: Quintic Newton-Schulz coefficients of the orthogonalised update.
COEFFS = (3.4445, -4.7750, 2.0315)
NS_EPS = 1e-7
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}


def listed():
    return [
        # the norm of a few sampled tokens while scoring online: latency
        {"name": "norm_few_tokens", "op": "norm", "dir": "fwd", "center": False, "n": 7, "d": 1024, "dtype": "bf16",
         "dy": "bf16", "wdtype": "bf16", "pad": 0, "eps": 1e-6},
        # scoring (no gradient) of a batch of rollouts in front of the LM head
        {"name": "norm_score", "op": "norm", "dir": "fwd", "center": False, "n": 8192, "d": 4096, "dtype": "bf16",
         "dy": "bf16", "wdtype": "bf16", "pad": 0, "eps": 1e-6},
        # the whole training batch: the LM head's backward hands down FP32 dhidden
        {"name": "norm_train_long", "op": "norm", "dir": "both", "center": False, "n": 32768, "d": 4096,
         "dtype": "bf16", "dy": "f32", "wdtype": "f32", "pad": 0, "eps": 1e-6},
        # layer norm with bias of an odd width, rows of a wider buffer
        {"name": "norm_odd_rows", "op": "norm", "dir": "both", "center": True, "n": 5003, "d": 1031, "dtype": "f16",
         "dy": "f16", "wdtype": "f16", "pad": 6, "eps": 1e-5},
        # one micro-batch: four pairs of short answers, prompts masked out
        {"name": "pref_micro", "op": "pref", "pairs": 4, "mean_len": 180, "kind": "sigmoid", "ref": True,
         "average": False, "beta": 0.1, "smooth": 0.0, "margin": 0.0, "masked": 0.3, "halves": False},
        # an ordinary batch, the chosen answers first, then the rejected ones
        {"name": "pref_batch", "op": "pref", "pairs": 128, "mean_len": 777, "kind": "sigmoid", "ref": True,
         "average": False, "beta": 0.05, "smooth": 0.1, "margin": 0.0, "masked": 0.25, "halves": True},
        # length-normalised reference-free form with a margin, ragged long answers
        {"name": "pref_no_reference", "op": "pref", "pairs": 501, "mean_len": 2500, "kind": "sigmoid", "ref": False,
         "average": True, "beta": 2.5, "smooth": 0.0, "margin": 1.0, "masked": 0.1, "halves": False},
        # 16.8 M tokens in 16384 sequences, the size of the policy-loss workload
        {"name": "pref_long", "op": "pref", "pairs": 8192, "mean_len": 1024, "kind": "ipo", "ref": True,
         "average": False, "beta": 0.1, "smooth": 0.0, "margin": 0.0, "masked": 0.25, "halves": True},
        # a small adapter's matrix: latency
        {"name": "orth_adapter", "op": "orth", "batch": 1, "m": 64, "n": 1024, "dtype": "bf16", "out": "bf16",
         "rank": 32, "steps": 5},
        # odd sizes, taller than wide, FP32 momentum
        {"name": "orth_tall_odd", "op": "orth", "batch": 1, "m": 2050, "n": 1001, "dtype": "f32", "out": "bf16",
         "rank": 100, "steps": 5},
        # a stack of equal matrices (one projection of several layers)
        {"name": "orth_stack", "op": "orth", "batch": 8, "m": 1024, "n": 4096, "dtype": "f32", "out": "bf16",
         "rank": 128, "steps": 5},
        # a square projection of the 4096-wide model
        {"name": "orth_square", "op": "orth", "batch": 1, "m": 4096, "n": 4096, "dtype": "f32", "out": "bf16",
         "rank": 512, "steps": 5},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "pref", "orth"])
    if op == "norm":
        d = _log(rng, 64, 8192)
        if rng.random() < 0.6:
            d = max(64, d // 64 * 64)
        n = _log(rng, 1, min(32768, 32768 * 4096 // d))
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        return {"op": op, "dir": rng.choice(["fwd", "both"]), "center": rng.random() < 0.5, "n": n, "d": d,
                "dtype": dtype, "dy": rng.choice([dtype, "f32"]), "wdtype": rng.choice([dtype, "f32"]),
                "pad": rng.choice([0, 0, 8, rng.randrange(1, 64)]), "eps": rng.choice([1e-5, 1e-6])}
    if op == "pref":
        pairs = _log(rng, 1, 8192)
        mean_len = _log(rng, 4, min(8192, 8192 * 1024 // pairs))
        kind = rng.choice(["sigmoid", "sigmoid", "ipo"])
        ref = rng.random() < 0.7
        return {"op": op, "pairs": pairs, "mean_len": mean_len, "kind": kind, "ref": ref, "average": not ref,
                "beta": rng.choice([0.05, 0.1, 0.3]) if ref else rng.choice([1.0, 2.0]),
                "smooth": rng.choice([0.0, 0.1]) if kind == "sigmoid" else 0.0,
                "margin": rng.choice([0.0, 0.5]) if kind == "sigmoid" else 0.0,
                "masked": rng.choice([0.0, 0.2, 0.5]), "halves": rng.random() < 0.5}
    a, b = _log(rng, 24, 4096), _log(rng, 24, 4096)
    if rng.random() < 0.6:
        a, b = max(8, a // 8 * 8), max(8, b // 8 * 8)
    lo = min(a, b)
    room = 4096.0 ** 3 / (float(lo) * a * b)
    return {"op": op, "batch": _log(rng, 1, max(1, min(16, int(room)))), "m": a, "n": b,
            "dtype": rng.choice(["bf16", "f32", "f32"]), "out": "bf16",
            "rank": max(1, lo // rng.choice([2, 4, 8])), "steps": rng.choice([5, 5, 6])}


# ---------------------------------------------------------------- inputs


def _norm_inputs(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 3 + 1)
    n, d, dt = c["n"], c["d"], DTYPES[c["dtype"]]

    def rows(dtype, make):
        buf = torch.zeros((n, d + c["pad"]), dtype=dtype, device="cuda")
        buf[:, :d] = make()
        return buf[:, :d]

    # hidden states: a per-row scale, a shift shared by the row and a few wide columns
    def hidden():
        h = torch.randn((n, d), generator=g, device="cuda")
        h *= torch.rand((n, 1), generator=g, device="cuda") * 1.5 + 0.5
        h[:, :: max(1, d // 7)] *= 6.0
        return h + 0.5 * torch.randn((n, 1), generator=g, device="cuda")

    s = {"x": rows(dt, hidden)}
    wdt = DTYPES[c["wdtype"]]
    s["weight"] = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(wdt)
    s["bias"] = (0.1 * torch.randn(d, generator=g, device="cuda")).to(wdt) if c["center"] else None
    if c["dir"] == "both":
        s["dy"] = rows(DTYPES[c["dy"]], lambda: torch.randn((n, d), generator=g, device="cuda") * 1e-2)
    return s


def _pref_inputs(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 3 + 2)
    seqs = 2 * c["pairs"]
    n = seqs * c["mean_len"]
    # ragged answers; now and then an empty one (a padded pair)
    share = torch.rand(seqs, generator=g, device="cuda", dtype=torch.float64) * 1.8 + 0.1
    share[torch.rand(seqs, generator=g, device="cuda") < 0.01] = 0
    share[0] = 1
    ends = torch.cumsum(share, 0)
    cu = torch.zeros(seqs + 1, dtype=torch.int64, device="cuda")
    cu[1:] = torch.round(ends / ends[-1] * n).to(torch.int64)
    logp = -torch.rand(n, generator=g, device="cuda") ** 3 * 8
    ref = logp + 0.2 * torch.randn(n, generator=g, device="cuda")
    mask = torch.rand(n, generator=g, device="cuda") >= c["masked"]
    # what a masked place holds has no meaning: some are -inf and NaN
    junk = ~mask & (torch.rand(n, generator=g, device="cuda") < 0.1)
    logp = torch.where(junk, torch.full_like(logp, -math.inf), logp)
    ref = torch.where(junk, torch.full_like(ref, math.nan), ref)
    return {"logp": logp, "ref": ref if c["ref"] else None, "cu": cu, "mask": mask}


def _orth_inputs(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 3 + 3)
    b, m, n, r = c["batch"], c["m"], c["n"], c["rank"]
    # a gradient: some directions with decaying strength over a noise floor
    s = torch.arange(1, r + 1, device="cuda", dtype=torch.float32).pow(-0.5)
    u = torch.randn((b, m, r), generator=g, device="cuda") * s
    v = torch.randn((b, r, n), generator=g, device="cuda")
    x = u @ v + 0.3 * torch.randn((b, m, n), generator=g, device="cuda")
    x = (x * 1e-3).to(DTYPES[c["dtype"]])
    return {"x": x[0] if b == 1 else x}


def prepare(case, seed):
    make = {"norm": _norm_inputs, "pref": _pref_inputs, "orth": _orth_inputs}[case["op"]]
    return {"case": case, **make(case, seed)}


# ---------------------------------------------------------------- plain forms


def _plain_norm(s):
    c, x = s["case"], s["x"].float()
    w = s["weight"].float()
    mean = x.mean(1, keepdim=True) if c["center"] else torch.zeros_like(x[:, :1])
    xc = x - mean
    rstd = torch.rsqrt((xc * xc).mean(1, keepdim=True) + c["eps"])
    xhat = xc * rstd
    y = xhat * w
    if s["bias"] is not None:
        y = y + s["bias"].float()
    out = {"y": y.to(s["x"].dtype)}
    if c["dir"] == "both":
        dy = s["dy"].float()
        gw = dy * w
        t = gw - xhat * (gw * xhat).mean(1, keepdim=True)
        if c["center"]:
            t = t - gw.mean(1, keepdim=True)
        out["dx"] = (t * rstd).to(s["x"].dtype)
        out["dweight"] = (dy * xhat).sum(0)
        out["dbias"] = dy.sum(0) if c["center"] else None
    return out


def _pairs_of(v, halves):
    """(chosen, rejected) of a per-sequence vector."""
    if halves:
        return v[: v.shape[0] // 2], v[v.shape[0] // 2:]
    return v[0::2], v[1::2]


def _plain_pref(s):
    c, logp, cu = s["case"], s["logp"], s["cu"]
    n, seqs = logp.shape[0], cu.shape[0] - 1
    beta = c["beta"]
    seq = torch.searchsorted(cu[1:], torch.arange(n, device=logp.device), right=True)
    d = logp if s["ref"] is None else logp - s["ref"]
    d = torch.where(s["mask"], d, torch.zeros_like(d))
    cnt = torch.zeros(seqs, device=logp.device).index_add_(0, seq, s["mask"].float())
    r = torch.zeros(seqs, device=logp.device).index_add_(0, seq, d)
    inv_len = 1 / cnt.clamp(min=1) if c["average"] else torch.ones_like(cnt)
    r = r * inv_len
    rc, rj = _pairs_of(r, c["halves"])
    cc, cj = _pairs_of(cnt, c["halves"])
    live = (cc > 0) & (cj > 0)
    h = rc - rj
    if c["kind"] == "sigmoid":
        u, e = beta * h - c["margin"], c["smooth"]
        each = (1 - e) * torch.log1p(torch.exp(-u.abs())) + e * torch.log1p(torch.exp(-u.abs()))
        each = each + (1 - e) * (-u).clamp(min=0) + e * u.clamp(min=0)
        dh = beta * (e / (1 + torch.exp(-u)) - (1 - e) / (1 + torch.exp(u)))
    else:
        t = h - 1 / (2 * beta)
        each, dh = t * t, 2 * t
    den = live.float().sum().clamp(min=1)
    loss = torch.where(live, each, torch.zeros_like(each)).sum() / den
    dh = torch.where(live, dh, torch.zeros_like(dh)) / den
    dr = torch.cat([dh, -dh]) if c["halves"] else torch.stack([dh, -dh], 1).reshape(-1)
    grad = torch.where(s["mask"], (dr * inv_len)[seq], torch.zeros_like(logp))
    return {"loss": loss.reshape(1), "grad": grad, "rewards": torch.stack([beta * rc, beta * rj], 1)}


def _plain_orth(s):
    c, x = s["case"], s["x"].float()
    a, b, k = COEFFS
    tall = c["m"] > c["n"]
    if tall:
        x = x.transpose(-1, -2)
    x = x / ((x * x).sum((-1, -2), keepdim=True).sqrt() + NS_EPS)
    for _ in range(c["steps"]):
        q = x @ x.transpose(-1, -2)
        x = a * x + (b * q + k * (q @ q)) @ x
    if tall:
        x = x.transpose(-1, -2)
    return {"update": x.to(DTYPES[c["out"]]).contiguous()}


# ---------------------------------------------------------------- the package's calls


def _own_norm(s):
    import selected_token_logprob_gb300 as flp

    c = s["case"]
    y, mean, rstd = flp.fused_layer_norm_forward(s["x"], s["weight"], s["bias"], eps=c["eps"], center=c["center"])
    out = {"y": y}
    if c["dir"] == "both":
        out["dx"], out["dweight"], out["dbias"] = flp.fused_layer_norm_backward(
            s["dy"], s["x"], s["weight"], mean, rstd, center=c["center"], with_dbias=c["center"])
    return out


def _own_pref(s):
    import selected_token_logprob_gb300 as flp

    c = s["case"]
    loss, grad, rewards = flp.logp_preference_loss(
        s["logp"], s["cu"], ref_logp=s["ref"], active_mask=s["mask"], kind=c["kind"], beta=c["beta"],
        label_smoothing=c["smooth"], margin=c["margin"], average=c["average"],
        layout="halves" if c["halves"] else "interleaved")
    return {"loss": loss, "grad": grad, "rewards": rewards}


def _own_orth(s):
    import selected_token_logprob_gb300 as flp

    c = s["case"]
    return {"update": flp.orthogonalize(s["x"], steps=c["steps"], coefficients=COEFFS, eps=NS_EPS,
                                        out_dtype=DTYPES[c["out"]])}


def run(state):
    forms = ({"norm": _own_norm, "pref": _own_pref, "orth": _own_orth} if own else
             {"norm": _plain_norm, "pref": _plain_pref, "orth": _plain_orth})
    return forms[state["case"]["op"]](state)


# ---------------------------------------------------------------- work


def work(case):
    c = case
    if c["op"] == "norm":
        n, d, e, w = c["n"], c["d"], BYTES[c["dtype"]], BYTES[c["wdtype"]]
        vecs = 2 if c["center"] else 1
        total = n * d * 2 * e + vecs * d * w
        if c["dir"] == "both":   # x, dy in, y, dx and the vectors' FP32 gradients out
            total = n * d * (3 * e + BYTES[c["dy"]]) + vecs * d * (w + 4)
        return {"bytes": total, "flops": n * d * (8 if c["dir"] == "fwd" else 20)}
    if c["op"] == "pref":
        n = 2 * c["pairs"] * c["mean_len"]
        return {"bytes": n * (4 + (4 if c["ref"] else 0) + 1 + 4) + 2 * c["pairs"] * (8 + 4),
                "flops": n * 3}
    lo, hi, b = min(c["m"], c["n"]), max(c["m"], c["n"]), c["batch"]
    # the two symmetric products cost half of a full one
    flops = c["steps"] * b * (float(lo) * lo * hi + float(lo) ** 3 + 2.0 * lo * lo * hi)
    return {"bytes": b * c["m"] * c["n"] * (BYTES[c["dtype"]] + BYTES[c["out"]]), "flops": flops}


# ---------------------------------------------------------------- values in 64 bits


def _exact_norm(s):
    c, f = s["case"], torch.float64
    x, w = s["x"].to(f), s["weight"].to(f)
    n, d = x.shape
    mu = x.sum(1) / d if c["center"] else torch.zeros(n, dtype=f, device=x.device)
    x = x - mu[:, None]
    sigma = torch.sqrt(torch.einsum("nd,nd->n", x, x) / d + c["eps"])
    x = x / sigma[:, None]
    y = torch.addcmul(s["bias"].to(f), x, w) if s["bias"] is not None else x * w
    out = {"y": y}
    if c["dir"] == "both":
        dy = s["dy"].to(f)
        out["dweight"] = torch.einsum("nd,nd->d", dy, x)
        out["dbias"] = dy.sum(0) if c["center"] else None
        v = dy * w
        out["dx"] = (v - (v.mean(1)[:, None] if c["center"] else 0)
                     - x * (torch.einsum("nd,nd->n", v, x) / d)[:, None]) / sigma[:, None]
    return out


def _exact_pref(s):
    import numpy as np

    c = s["case"]
    logp, cu, mask = s["logp"].double().cpu().numpy(), s["cu"].cpu().numpy(), s["mask"].cpu().numpy()
    d = logp if s["ref"] is None else logp - s["ref"].double().cpu().numpy()
    d = np.where(mask, d, 0.0)
    seqs, beta = len(cu) - 1, float(c["beta"])
    cnt, r = np.zeros(seqs), np.zeros(seqs)
    for k in range(seqs):
        cnt[k] = mask[cu[k]: cu[k + 1]].sum()
        r[k] = d[cu[k]: cu[k + 1]].sum()
    scale = 1 / np.maximum(cnt, 1) if c["average"] else np.ones(seqs)
    r = r * scale
    chosen = np.arange(seqs // 2) if c["halves"] else np.arange(0, seqs, 2)
    rejected = chosen + (seqs // 2 if c["halves"] else 1)
    live = (cnt[chosen] > 0) & (cnt[rejected] > 0)
    h = r[chosen] - r[rejected]
    if c["kind"] == "sigmoid":
        u, e = beta * h - c["margin"], c["smooth"]
        each = (1 - e) * np.logaddexp(0, -u) + e * np.logaddexp(0, u)
        dh = beta * (np.exp(-np.logaddexp(0, -u)) - (1 - e))
    else:
        each = (h - 0.5 / beta) ** 2
        dh = 2 * (h - 0.5 / beta)
    den = max(1, int(live.sum()))
    dr = np.zeros(seqs)
    dr[chosen] = np.where(live, dh, 0) / den
    dr[rejected] = -dr[chosen]
    grad = np.where(mask, np.repeat(dr * scale, np.diff(cu)), 0.0)
    return {"loss": np.array([np.where(live, each, 0).sum() / den]), "grad": grad,
            "rewards": beta * np.stack([r[chosen], r[rejected]], 1)}


def _exact_orth(s):
    c = s["case"]
    a, b, k = COEFFS
    x = s["x"].double()
    x = x / (torch.linalg.vector_norm(x, dim=(-2, -1), keepdim=True) + NS_EPS)
    for _ in range(c["steps"]):
        # p(x) = x (a + b q + k q^2) on the smaller side, by Horner's rule
        tall = x.shape[-2] > x.shape[-1]
        q = x.mT @ x if tall else x @ x.mT
        p = k * q
        p.diagonal(dim1=-2, dim2=-1).add_(b)
        p = p @ q
        p.diagonal(dim1=-2, dim2=-1).add_(a)
        x = x @ p if tall else p @ x
    return {"update": x.contiguous()}


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "pref": _exact_pref, "orth": _exact_orth}[case["op"]](s)
