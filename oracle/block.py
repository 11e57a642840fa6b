"""fp64 CPU oracle of the gated linear recurrence, the log probabilities of tokens and the gated
feed-forward block.

TEST INFRASTRUCTURE ONLY, like the rest of this package: it shares no code with the HIP library
and imports nothing from the product package.

Everything is float64 and follows the definitions line by line:

* recurrence: r = sigmoid(ga), i = sigmoid(gx), a = exp(lam r), m = sqrt(1 - a^2),
  h_t = a_t h_{t-1} + m_t i_t x_t
* log probabilities: log softmax(scale x) at the ids, its entropy, the likeliest columns
* feed-forward: act(x Wg^T) * (x Wu^T)

The gradients are the chain rule of these, by hand.  Beside a result, its ``err`` is a bound on
the error of a computation in fp32, in units of the unit roundoff, from the roundings of every
step carried through the recurrence (first order).
"""
from __future__ import annotations

import numpy as np


def _f64(a):
    return None if a is None else np.asarray(a, dtype=np.float64)


def sigmoid(z):
    e = np.exp(-np.abs(z))
    return np.where(z >= 0, 1.0, e) / (1.0 + e)


# ---- the gated linear recurrence -----------------------------------------------------------

# Roundings, in units of the roundoff.  sigmoid(g): the exponent g log2 e is off by 2 |g|, the exp,
# the sum and the reciprocal by 2, 1 and 2.  a = exp(lam r): the exponent's error times its size,
# and 4.  m: half of that of 1 - a^2, whose series keeps the relative error of q and whose
# difference (from q = 0.4 on) at most doubles it; with the root and its products, 16 more.  The
# compositions add at most 8 + 6 + 6 + 4 steps one after another, two roundings each.
def _step_errors(ga, gx, la):
    ea = np.abs(la) * (2 * np.abs(ga) + 8) + 4
    eb = 2 * np.abs(ga) + 2 * np.abs(gx) + 32
    return ea + 48, eb + 48


def lru_fwd(x, ga, gx, lam, h0=None):
    """dict of out [batch, dim, seqlen] and final, with their err."""
    x, ga, gx, lam = map(_f64, (x, ga, gx, lam))
    la = lam[None, :, None] * sigmoid(ga)
    a, m = np.exp(la), np.sqrt(-np.expm1(2 * la))
    b = m * sigmoid(gx) * x
    ea, eb = _step_errors(ga, gx, la)
    h = np.zeros(x.shape[:2]) if h0 is None else _f64(h0).copy()
    err = np.zeros_like(h)
    out, errs = np.empty_like(x), np.empty_like(x)
    for t in range(x.shape[2]):
        err = a[..., t] * err + ea[..., t] * a[..., t] * np.abs(h) + eb[..., t] * np.abs(b[..., t])
        h = a[..., t] * h + b[..., t]
        out[..., t], errs[..., t] = h, err
    return dict(out=out, out_err=errs, final=h, final_err=err)


def lru_bwd(x, ga, gx, lam, dout, h0=None, dfinal=None):
    """dict of dx, dga, dgx, dlam, dh0, with their err."""
    f = lru_fwd(x, ga, gx, lam, h0)
    x, ga, gx, lam, dout = map(_f64, (x, ga, gx, lam, dout))
    lam = lam[None, :, None]
    r, i = sigmoid(ga), sigmoid(gx)
    la = lam * r
    a, m = np.exp(la), np.sqrt(-np.expm1(2 * la))
    ea, eb = _step_errors(ga, gx, la)
    first = np.zeros(x.shape[:2]) if h0 is None else _f64(h0)
    before = np.concatenate([first[..., None], f["out"][..., :-1]], -1)
    before_err = np.concatenate([0 * first[..., None], f["out_err"][..., :-1]], -1)
    g, gerr = np.empty_like(x), np.empty_like(x)
    e = np.zeros_like(first) if dfinal is None else _f64(dfinal).copy()
    err = np.zeros_like(e)
    for t in range(x.shape[2] - 1, -1, -1):
        g[..., t] = dout[..., t] + e
        gerr[..., t] = err + np.abs(dout[..., t]) + np.abs(e)
        e = a[..., t] * g[..., t]
        err = a[..., t] * gerr[..., t] + ea[..., t] * np.abs(e)
    slope = np.divide(i * x * a * a, m, out=np.zeros_like(x), where=m > 0)
    q = g * (a * before - slope)
    qterms = np.abs(g) * (a * np.abs(before) + np.abs(slope))
    qerr = (gerr * np.abs(a * before - slope) + np.abs(g) * a * before_err + (ea + eb) * qterms)
    gm = g * m
    gmerr = gerr * m + eb * np.abs(gm)
    more = 2 * np.abs(ga) + 2 * np.abs(gx) + 32
    dga, dgx, dx = q * lam * r * (1 - r), gm * x * i * (1 - i), gm * i
    return dict(dx=dx, dx_err=gmerr * i + more * np.abs(dx),
                dga=dga, dga_err=qerr * np.abs(lam) * r * (1 - r)
                + (more + 4 / np.maximum(1 - r, 1e-9)) * qterms * np.abs(lam) * r * (1 - r),
                dgx=dgx, dgx_err=gmerr * np.abs(x) * i * (1 - i)
                + (more + 4 / np.maximum(1 - i, 1e-9)) * np.abs(dgx),
                dlam=(q * r).sum((0, 2)),
                dlam_err=(qerr * r + (more + 128) * qterms * r).sum((0, 2)),
                dh0=e, dh0_err=err)


# ---- log probabilities ---------------------------------------------------------------------

def logprob_fwd(logits, ids=None, scale=1.0, top=0):
    """dict of lse, entropy, logprob (with ids), top_ids and top_logprobs, and p; err in units of
    the roundoff, for sums whose terms are added at most 64 + vocab / 256 one after another."""
    raw = _f64(logits)
    x = raw * scale
    m = x.max(-1, keepdims=True)
    m = np.where(np.isinf(m), 0.0, m)
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.exp(x - m)
        s = e.sum(-1, keepdims=True)
        dead = s[..., 0] == 0
        lse = (m + np.log(s))[..., 0]
        p = np.where(s > 0, e / np.where(s > 0, s, 1.0), 0.0)
        lp = np.where(dead[..., None], -np.inf, x - lse[..., None])
    d = np.where(p > 0, x - m, 0.0)
    spread = (p * np.abs(d)).sum(-1)
    adds = 64 + raw.shape[-1] / 256
    sum_err = 2 * spread + adds
    log_s = np.where(dead, 0.0, lse - m[..., 0])
    out = dict(lse=lse, p=p, lp=lp, dead=dead, sum_err=sum_err,
               lse_err=2 * np.abs(m[..., 0]) + 2 * np.abs(log_s) + sum_err,
               entropy=np.where(dead, 0.0, log_s - (p * d).sum(-1)),
               entropy_err=2 * np.abs(log_s) + sum_err
               + (p * np.abs(d) * (2 * np.abs(d) + adds + 4)).sum(-1) + spread * (sum_err + 4))
    if ids is not None:
        ids = np.asarray(ids)
        real = (ids >= 0) & (ids < raw.shape[-1])
        at = np.where(real, ids, 0)[..., None]
        out["logprob"] = np.where(real, np.take_along_axis(lp, at, -1)[..., 0], 0.0)
        far = np.abs(np.take_along_axis(np.where(np.isinf(x), m, x), at, -1) - m)[..., 0]
        out["logprob_err"] = 4 * far + 2 * np.abs(log_s) + sum_err
    if top:
        order = np.argsort(-raw, axis=-1, kind="stable")[..., :top]
        out["top_ids"] = order
        out["top_logprobs"] = np.take_along_axis(lp, order, -1)
        far = np.abs(np.take_along_axis(np.where(np.isinf(x), m, x), order, -1) - m)
        out["top_err"] = 4 * far + (2 * np.abs(log_s) + sum_err)[..., None]
    return out


def logprob_bwd(logits, ids, scale=1.0, dlogprob=None, dlse=None, dentropy=None):
    """dlogits and its err.  The roundings of log p: those of scale x, of lse and of the given lse
    and entropy, times p."""
    f = logprob_fwd(logits, ids, scale)
    p, lp = f["p"], np.where(f["p"] > 0, f["lp"], 0.0)
    x = np.where(np.isinf(_f64(logits)), 0.0, _f64(logits) * scale)
    zero = np.zeros(p.shape[:-1])
    dlp, dl, dh = (zero if v is None else _f64(v) for v in (dlogprob, dlse, dentropy))
    real = (np.asarray(ids) >= 0) & (np.asarray(ids) < p.shape[-1]) if ids is not None else zero > 0
    dlp = np.where(real, dlp, 0.0)
    lse = np.where(f["dead"], 0.0, f["lse"])
    H = f["entropy"][..., None]
    c = (dl - dlp)[..., None] - dh[..., None] * (lp + H)
    d = p * c
    np.put_along_axis(d, np.where(real, ids if ids is not None else 0, 0)[..., None].astype(int),
                      np.take_along_axis(d, np.where(real, ids if ids is not None else 0, 0)
                                         [..., None].astype(int), -1) + dlp[..., None], -1)
    d = np.where(f["dead"][..., None], 0.0, d * scale)
    # log p is off by the roundings of scale x, of lse and of their difference; that of a given
    # fp32 entropy and lse as well
    loge = 2 * np.abs(x) + (3 * np.abs(lse) + f["lse_err"])[..., None] + 4
    terms = np.abs(dl - dlp)[..., None] + np.abs(dh)[..., None] * (np.abs(lp) + np.abs(H))
    err = scale * (p * (terms * (loge + 8) + np.abs(dh)[..., None]
                        * (loge + f["entropy_err"][..., None])) + 2 * np.abs(d) / scale)
    return d, err


# ---- the gated feed-forward block ----------------------------------------------------------

def act(z, gelu):
    """(act(z), act'(z))."""
    if not gelu:
        s = sigmoid(z)
        return z * s, s * (1 + z * (1 - s))
    c = np.sqrt(2 / np.pi)
    t = np.tanh(c * (z + 0.044715 * z ** 3))
    return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 0.134145 * z * z)


def mlp_fwd(x, wg, wu, gelu=False):
    x, wg, wu = map(_f64, (x, wg, wu))
    return act(x @ wg.T, gelu)[0] * (x @ wu.T)


def mlp_bwd(x, wg, wu, dout, gelu=False):
    """dict of dx, dwg, dwu and the inner dg, du."""
    x, wg, wu, dout = map(_f64, (x, wg, wu, dout))
    v, slope = act(x @ wg.T, gelu)
    dg, du = dout * (x @ wu.T) * slope, dout * v
    return dict(dx=dg @ wg + du @ wu, dwg=dg.T @ x, dwu=du.T @ x, dg=dg, du=du)
