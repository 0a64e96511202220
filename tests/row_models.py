"""Error models of the row operators (layer norm, token log probabilities, distillation) and
the comparison that uses them (test infrastructure).

Every bound is |gpu - ref| <= half * |ref| + E: ``half`` is half a step of the output's type
(one rounding to nearest) and E the rounding model of a correct fp32 evaluation, written out
per operator below with u = 2^-24.  Sums along a row run as a tree over lanes whose longest
chain is taken as 96 additions (G = 96 u times the magnitude sum); column sums over many rows
take 2^-16 times the magnitude sum, as the bias gradients do.
"""
from __future__ import annotations

import numpy as np
import torch

from parity import FP16_SUBNORMAL_HALF, TORCH_NAME, sum_abs_model, to64

U = 2.0 ** -24
G = 96 * U
FLOOR = {"bf16": 2.0 ** -126, "fp16": FP16_SUBNORMAL_HALF, "fp32": 2.0 ** -126}


def check(name, got, ref, model):
    """Element by element, infinities and NaN in the same places."""
    half = torch.finfo(got.dtype).eps / 2
    floor = FLOOR[TORCH_NAME[got.dtype]]
    g, r = to64(got), np.asarray(ref, dtype=np.float64)
    assert g.shape == r.shape, f"{name}: shape {g.shape}, expected {r.shape}"
    fin = np.isfinite(r)
    # a finite value beyond the type's range rounds to infinity
    big = float(torch.finfo(got.dtype).max)
    over = fin & (np.abs(r) > big)
    assert np.array_equal(np.isnan(g), np.isnan(r)), f"{name}: NaN in other places"
    same = np.isinf(r)
    assert np.array_equal(g[same], r[same]), f"{name}: infinities differ"
    m = fin & ~over
    model = np.broadcast_to(np.asarray(model, dtype=np.float64), r.shape)
    err = np.abs(g[m] - r[m])
    bound = half * np.abs(r[m]) + model[m] + floor
    bad = ~(err <= bound)
    if bad.any():
        i = int(np.argmax(np.where(bad, err / bound, 0)))
        raise AssertionError(f"{name}: {int(bad.sum())} of {r.size} outside the bound; worst "
                             f"gpu {g[m][i]!r} ref {r[m][i]!r} bound {bound[i]:.3g}")


def norm_models(x, w, mean, rstd):
    """(y, mean, rstd) models.  err_d: a centred value x - mean, from the mean's tree and the
    subtraction."""
    x = to64(x)
    aw = 1.0 if w is None else np.abs(to64(w))
    mag = np.abs(x).mean(1)
    e_mean = G * mag + 2 * U * np.abs(mean)
    e_d = e_mean[:, None] + U * (np.abs(x) + np.abs(mean)[:, None])
    # var is a mean of d^2: its relative error is the tree's plus twice the relative error of
    # the d (root mean square over the row); the root halves it
    rel = G + 4 * U + np.sqrt((e_d * e_d).mean(1)) * rstd
    xh = (x - mean[:, None]) * rstd[:, None]
    e_y = aw * (rstd[:, None] * e_d + np.abs(xh) * (rel[:, None] + 4 * U))
    return e_y + 2 * U * np.abs(xh) * aw, e_mean, rstd * rel


def norm_bwd_models(dy, x, w, mean, rstd, dw0=None, db0=None):
    """(dx, dw, db) models, statistics taken as given."""
    dy, x = to64(dy), to64(x)
    mu, rs = to64(mean)[:, None], to64(rstd)[:, None]
    xh = (x - mu) * rs
    e_xh = rs * U * (np.abs(x) + np.abs(mu)) + 2 * U * np.abs(xh)
    h = np.abs(dy if w is None else dy * to64(w))
    c1 = h.mean(1, keepdims=True)
    c2 = (h * np.abs(xh)).mean(1, keepdims=True)
    e_c2 = (G + 2 * U) * c2 + (h * e_xh).mean(1, keepdims=True)
    e_dx = rs * (2 * U * h + (G + U) * c1 + np.abs(xh) * e_c2 + e_xh * c2
                 + 4 * U * (h + c1 + np.abs(xh) * c2))
    e_dw = sum_abs_model((np.abs(dy) * np.abs(xh)).sum(0)) + (np.abs(dy) * e_xh).sum(0)
    e_db = sum_abs_model(np.abs(dy).sum(0))
    for e, init in ((e_dw, dw0), (e_db, db0)):
        if init is not None:
            e += U * np.abs(to64(init))
    return e_dx, e_dw, e_db


def _finite_max(a):
    b = np.where(np.isfinite(a), np.abs(a), 0.0)
    return b.max(1, keepdims=True)


def logit_errors(z, t, lp, lse):
    """Absolute error of a log probability (and relative error of a probability): the scaled
    logit (2 u |a|), the row's largest one (the same), the sum of exponentials (G, each
    exponential 4 u) and the roundings of lse and of the difference."""
    a = to64(z) / t
    al = np.where(np.isfinite(lse), np.abs(lse), 0.0)[:, None]
    alp = np.where(np.isfinite(lp), np.abs(lp), 0.0)
    return G + 8 * U + U * (4 * _finite_max(a) + 2 * al + 4 * alp)


def entropy_model(lp, d):
    p = np.exp(lp)
    alp = np.where(np.isfinite(lp), np.abs(lp), 0.0)
    h = (p * alp).sum(1)
    return (p * (alp + 1) * d).sum(1) + G * (1 + h)


def logprobs_bwd_model(t, lp, d, g, h, entropy):
    p = np.exp(lp)
    alp = np.where(np.isfinite(lp), np.abs(lp), 0.0)
    g, h, ent = np.abs(g)[:, None], np.abs(h)[:, None], np.abs(entropy)[:, None]
    e = g * p * (d + 4 * U) + h * p * ((alp + ent + 1) * d + 8 * U * (alp + ent))
    return (e + 4 * U * g * (p + (p > 0.5))) / t


def teacher_errors(u, t, lq):
    """Absolute error of a teacher's log probability, as ``logit_errors``."""
    a = np.where(np.isfinite(lq), to64(u) / t, 0.0)
    alq = np.where(np.isfinite(lq), np.abs(lq), 0.0)
    return G + 8 * U + U * (6 * np.abs(a).max(1, keepdims=True) + 4 * alq)


def distill_model(t, lq, q, lp_at, d_at, dq):
    diff = np.where(q > 0, np.abs(lq - lp_at), 0.0)
    diff = np.where(np.isfinite(diff), diff, 0.0)
    e = (q * (diff * (dq + 8 * U) + dq + d_at)).sum(1)
    return t * t * (e + G * (q * diff).sum(1))


def distill_bwd_model(z, t, ids, p, d, q, dq, c):
    """Each column's share of the teacher is a sum over its entries."""
    V = z.shape[1]
    e = p * (d + 8 * U)
    for r in range(z.shape[0]):
        np.add.at(e[r], np.clip(ids[r], 0, V - 1), q[r] * (dq[r] + G))
    return np.abs(c)[:, None] * t * e
