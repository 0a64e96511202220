"""Error models of the residual norm (see row_models for their form)."""
from __future__ import annotations

import numpy as np

from parity import sum_abs_model, to64
from row_models import G, U


def _mag(t, like):
    return np.ones_like(like) if t is None else np.abs(np.broadcast_to(to64(t), like.shape))


def fwd_models(y, residual, w_post, w_pre, gate, scale, rs, rp, out):
    """(out, norm, rstd_post, rstd_pre) models; rs, rp and out are the reference's."""
    y = to64(y)
    rel = G + 4 * U                       # of a root: half its sum's tree, and its own roundings
    u = np.abs(y) if rs is None else np.abs(y) * rs[:, None] * _mag(w_post, y)
    part = abs(scale) * u * _mag(gate, y)
    e_out = part * (rel + 8 * U) + 2 * U * np.abs(out)
    e_rs = None if rs is None else rs * rel
    if rp is None:
        return e_out, None, e_rs, None
    rel_p = rel + np.sqrt((e_out * e_out).mean(1)) * rp
    r = rp[:, None]
    e_norm = _mag(w_pre, y) * r * (e_out + np.abs(out) * (rel_p[:, None] + 4 * U))
    return e_out, e_norm, e_rs, rp * rel_p


def bwd_models(dout, dnorm, y, out, w_post, w_pre, gate, rstd_post, rstd_pre, scale):
    """(dy, dresidual, dw_post, dw_pre, dgate) models with the statistics as given."""
    y = to64(y)
    zero = np.zeros_like(y)
    d = zero if dout is None else np.abs(to64(dout))
    rp = 0.0 if rstd_pre is None or dnorm is None else to64(rstd_pre)[:, None]
    dn = zero if dnorm is None else np.abs(to64(dnorm))
    xh = zero if dnorm is None else np.abs(to64(out)) * rp
    h = dn * _mag(w_pre, y)
    c = (h * xh).mean(1, keepdims=True)
    e_c = (G + 6 * U) * c
    D = d + rp * (h + xh * c)
    e_D = 6 * U * D + rp * xh * e_c
    rs = 1.0 if rstd_post is None else to64(rstd_post)[:, None]
    yh = np.abs(y) * rs
    u = yh * _mag(None if rstd_post is None else w_post, y)
    row = gate is not None and np.ndim(gate) == 2 and np.shape(gate)[1] == 1 != y.shape[1]
    g = _mag(gate, y)
    ye = u * (1.0 if row else g)
    k = abs(scale) * (g[:, :1] if row else 1.0)
    tail = rp * (xh * ye).mean(1, keepdims=True)
    t = ((d + rp * h) * ye).mean(1, keepdims=True) + c * tail
    e_t = (G + 8 * U) * t + e_c * tail
    if rstd_post is None:
        e_dy = abs(scale) * g * (e_D + 4 * U * D)
    else:
        e = _mag(w_post, y) * (1.0 if row else g)
        e_dy = rs * k * (e * e_D + yh * e_t + 8 * U * (e * D + yh * t))
    gd = abs(scale) * g * D
    e_dwp = sum_abs_model((gd * yh).sum(0)) + (abs(scale) * g * yh * (e_D + 6 * U * D)).sum(0)
    e_dwq = sum_abs_model((dn * xh).sum(0)) + (4 * U * dn * xh).sum(0)
    e_dg = abs(scale) * u * (e_D + 6 * U * D)
    if row:
        e_dg = abs(scale) * y.shape[1] * e_t
    elif gate is not None and np.ndim(gate) == 1:
        e_dg = e_dg.sum(0) + sum_abs_model(abs(scale) * (D * u).sum(0))
    return e_dy, e_D, e_dwp, e_dwq, e_dg
