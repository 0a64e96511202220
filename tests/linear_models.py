"""Error models of the linear layer (see row_models for their form)."""
from __future__ import annotations

import numpy as np
import torch

from parity import sum_abs_model, to64
from row_models import U


def fwd_models(x, w, bias, residual, act, y, z):
    """(y, z) models; y and z are the reference's.  An activation moves by at most 1.2 times its
    argument's error (the largest slope of z sigma(beta z), 1.1 whatever beta, and of gelu, 1.13)
    and is itself within 64 roundings of its argument."""
    mag = np.abs(to64(x)) @ np.abs(to64(w))
    if bias is not None:
        mag = mag + np.abs(to64(bias))
    e_z = sum_abs_model(mag)
    e_y = e_z
    if act != "none":
        e_y = 1.2 * e_z + 64 * U * np.abs(z)
    res = 0.0 if residual is None else np.abs(to64(residual))
    return e_y + 2 * U * (np.abs(y) + 2 * res), e_z


def bwd_models(dy, x, w, z, act, dz):
    """(dx, dw, db) models; dz is the reference's.  dz is rounded to the operands' type (half a
    step) and its slope is within 64 roundings of 1 + |z|."""
    dy = to64(dy)
    half = torch.finfo(x.dtype).eps / 2
    slope = 0.0 if act == "none" else np.abs(dy) * 64 * U * (1 + np.abs(to64(z)))
    # values under the smallest normal number lose their relative precision
    e_dz = slope if act == "none" else slope + half * (np.abs(dz) + torch.finfo(x.dtype).tiny)
    aw, ax, ad = np.abs(to64(w)), np.abs(to64(x)), np.abs(dz)
    e_dx = sum_abs_model(ad @ aw.T)
    e_dw = sum_abs_model(ax.T @ ad)
    e_db = sum_abs_model(ad.sum(0))
    if act != "none":
        e_dx = e_dx + e_dz @ aw.T
        e_dw = e_dw + ax.T @ e_dz
        e_db = e_db + slope.sum(0)
    return e_dx, e_dw, e_db
