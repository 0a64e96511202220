"""Error models whose bounds do not grow with the size of the logits (test infrastructure).

The operators form z - m for the row's largest logit m before they scale, so a log probability's
error follows its own size |lp| (every |z - m| / T is at most |lp|: log sum exp (a - m) >= 0) and
the entropy H (which bounds sum p |a - m| and log sum exp (a - m)), not |a|.  With u = 2^-24:
3 u |lp| for the difference, 1 / T and the product, u for the last subtraction; the sum of
exponentials G, each exponential 2 u and 5 u of its exponent (log2 e / T is rounded three times);
2 u of the logarithm.  8 u (|lp| + H) + 16 u + G covers them.
"""
from __future__ import annotations

import numpy as np

import oracle.ref as R
from parity import to64
from row_models import G, U, check, distill_bwd_model, distill_model, entropy_model


def log_softmax(z, T):
    """(log p, lse) from the differences z - m: a log sum exp beside a large m / T would be
    rounded off in float64 too.  z = -inf has log p = -inf; a row of nothing else has lse = -inf
    and log p = -inf."""
    m = z.max(1, keepdims=True)
    empty = np.isneginf(m)
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        d = np.where(np.isneginf(z), -np.inf, (z - np.where(empty, 0.0, m)) / T)
        ls = np.log(np.exp(d).sum(1, keepdims=True))
        lp = np.where(np.isneginf(d), -np.inf, d - np.where(empty, 0.0, ls))
        return lp, np.where(empty, -np.inf, m / T + ls)[:, 0]


def row_errors(lp):
    """Absolute error of a log probability, relative error of a probability."""
    alp = np.where(np.isfinite(lp), np.abs(lp), 0.0)
    return G + 16 * U + 8 * U * (alp + R.entropy_ref(lp)[:, None])


def lse_errors(z64, T, lp, lse):
    """m / T (two roundings) + log sum exp (a - m)."""
    m = np.where(np.isfinite(z64), z64, -np.inf).max(1)
    m = np.where(np.isfinite(m), np.abs(m), 0.0) / T
    al = np.where(np.isfinite(lse), np.abs(lse), 0.0)
    return row_errors(lp).min(1) + U * (2 * m + al)


def entropy_errors(lp):
    return entropy_model(lp, row_errors(lp))


def teacher_row_errors(lq):
    alq = np.where(np.isfinite(lq), np.abs(lq), 0.0)
    return G + 16 * U + 8 * U * alq


def check_forward(z, t, r, T, top):
    """logprob, entropy, lse and the top entries of every row."""
    T, z64 = float(np.float32(T)), to64(z)
    lp, lse = log_softmax(z64, T)
    d = row_errors(lp)
    check("lse", r.lse, lse, lse_errors(z64, T, lp, lse))
    check("entropy", r.entropy, R.entropy_ref(lp), entropy_errors(lp))
    if t is not None:
        rows, at = np.arange(len(t)), t.cpu().numpy()
        check("logprob", r.logprob, lp[rows, at], d[rows, at])
    if top:
        ids = R.top_ref(z64, top)
        assert np.array_equal(r.top_id.cpu().numpy(), ids), "top_id"
        check("top_logprob", r.top_logprob, np.take_along_axis(lp, ids, 1),
              np.take_along_axis(d, ids, 1))


def check_loss(z, u, ids, T, loss, lse, c=None, dz=None):
    """Loss and lse, and with ``dz`` the gradient of the one-call form (p from m and the log
    sum)."""
    T, z64, idn = float(np.float32(T)), to64(z), ids.cpu().numpy()
    V = z64.shape[1]
    lp, ref_lse = log_softmax(z64, T)
    lq, _ = log_softmax(np.where((idn >= 0) & (idn < V), to64(u), -np.inf), T)
    q = np.exp(lq)
    d, dq = row_errors(lp), teacher_row_errors(lq)
    at = np.clip(idn, 0, V - 1)
    lp_at = np.take_along_axis(lp, at, 1)
    with np.errstate(invalid="ignore"):
        ref = T * T * np.where(q > 0, q * (lq - lp_at), 0.0).sum(1)
    check("loss", loss, ref,
          distill_model(T, lq, q, lp_at, np.take_along_axis(d, at, 1), dq))
    check("lse", lse, ref_lse, lse_errors(z64, T, lp, ref_lse))
    if dz is not None:
        cn = to64(c)
        p = np.exp(lp)
        e = p * (q.sum(1, keepdims=True) > 0)
        for r in range(len(e)):
            np.subtract.at(e[r], at[r], q[r])
        check("dlogits", dz, cn[:, None] * T * e,
              distill_bwd_model(z64, T, idn, p, d, q, dq, cn))
