"""Plain float64 CPU oracle for the SwiGLU backward and the beta-scaled Swish gradient, layer
norm, token log probabilities and distillation from a teacher's top logits.

TEST INFRASTRUCTURE ONLY.  Nothing in the product path may import, call or run this
module: only the tests, the package's smoke check and the bench's CPU-baseline leg use
it.  It shares no code with the HIP kernels or their host library.

Every function is the plain mathematical definition written out in numpy float64,
with no blocking, fusion or reordering.  Inputs are the exact tensors the GPU
received, widened to float64 (exact for bf16, fp16 and fp32).  Sources:

  [SwiGLU page]  "PyPTO-Gym 实战: Fused SwiGLU 反向传播算子" (hnwysp.cn), section
                 "算法概述与数学公式" (algorithm overview and formulas), items 1-4,
                 and the SwiGLU forward in "算子背景" (operator background).
  [Swish page]   "CANN ops-nn 中 SwishGrad 算子解析" (bhfrc.com), section 1.2
                 "计算公式" (formula) and section 2.4 (kernel compute chain).
  [Ascend C page] "Ascend C 自定义反向算子" (cann.csdn.net), section 2.1 (math
                 definition of the Swish gradient).

Readings taken where the pages are garbled or silent:
  * The SwiGLU page's extracted formulas lost '=', '+' and the prime on SiLU'.  The
    gate gradient is read as dg = dy*fc*SiLU'(g) with SiLU'(g) = s(1 + g(1 - s)),
    s = sigmoid(g); the page's description of its code builds dg the same way (the
    product dy*fc times the SiLU derivative), and it is the derivative of g*sigmoid(g).
  * The sigmoid is 1/(1 + exp(-t)) (the Swish page's definition), which is finite for
    every finite t; the SwiGLU page's exp(g)/(1 + exp(g)) is the same function.
  * db and dw are accumulated into caller-provided buffers (the SwiGLU page says they
    must be zero-initialised because the kernels add into them); the oracle adds the
    initial value exactly.
  * beta is a float32 scalar on the Swish page; the oracle widens that float32 value.
"""
from __future__ import annotations

import numpy as np

__all__ = ["sigmoid", "silu", "silu_grad", "swish_grad_ref", "b_ref", "w_ref",
           "x_ref", "swiglu_forward_ref", "swiglu_bwd_ref", "layer_norm_ref",
           "layer_norm_bwd_ref", "log_softmax_ref", "entropy_ref", "top_ref",
           "token_logprobs_bwd_ref", "teacher_ref", "distill_ref", "distill_bwd_ref"]


def _f64(a) -> np.ndarray:
    return np.asarray(a, dtype=np.float64)


def sigmoid(t):
    """sigma(t) = 1 / (1 + exp(-t))  [Swish page, section 1.2, sigmoid definition].

    exp(-t) overflows to +inf for t < -709; 1/(1+inf) = 0 is then the correct limit.
    """
    t = _f64(t)
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-t))


def silu(t):
    """SiLU(t) = t * sigma(t)  [SwiGLU page, operator background]."""
    t = _f64(t)
    return t * sigmoid(t)


def silu_grad(t):
    """d/dt SiLU(t) = sigma(t) * (1 + t * (1 - sigma(t)))  [SwiGLU page, formula 1]."""
    t = _f64(t)
    s = sigmoid(t)
    return s * (1.0 + t * (1.0 - s))


def swish_grad_ref(grad, x, beta=1.0):
    """grad_x = grad * s'(x),  s(x) = x * sigma(beta x),
    s'(x) = sigma(beta x) * (1 + beta x * (1 - sigma(beta x)))
    [Swish page, section 1.2, derivative of the Swish forward; Ascend C page, 2.1].

    ``beta`` is the float32 scalar the kernel receives (None means 1.0, as the Swish
    page's aclnn interface specifies for a missing beta).
    """
    b = 1.0 if beta is None else float(np.float32(beta))
    x = _f64(x)
    t = b * x
    s = sigmoid(t)
    return _f64(grad) * (s * (1.0 + t * (1.0 - s)))


def b_ref(dy, g, fc, db_g0=None, db_fc0=None):
    """b stage [SwiGLU page, formulas 1 and 2]:
        dg  = dy * fc * SiLU'(g)
        dfc = dy * SiLU(g) = dy * g * sigma(g)
        db_g  = db_g0  + sum over the batch dimension of dg
        db_fc = db_fc0 + sum over the batch dimension of dfc
    dy, g, fc: [M, N].  Returns (dg, dfc, db_g, db_fc) in float64.
    """
    dy, g, fc = _f64(dy), _f64(g), _f64(fc)
    N = dy.shape[-1]
    dg = dy * fc * silu_grad(g)
    dfc = dy * silu(g)
    db_g = (np.zeros(N) if db_g0 is None else _f64(db_g0).reshape(N)) + dg.sum(axis=0)
    db_fc = (np.zeros(N) if db_fc0 is None else _f64(db_fc0).reshape(N)) + dfc.sum(axis=0)
    return dg, dfc, db_g, db_fc


def w_ref(x, dg, dfc, dw_g0=None, dw_fc0=None):
    """w stage [SwiGLU page, formula 3]: dw_g = dw_g0 + x^T dg, dw_fc = dw_fc0 + x^T dfc.

    x: [M, K]; dg, dfc: [M, N].  Returns (dw_g, dw_fc), each [K, N] float64.
    """
    x, dg, dfc = _f64(x), _f64(dg), _f64(dfc)
    K, N = x.shape[1], dg.shape[1]
    dw_g = x.T @ dg
    dw_fc = x.T @ dfc
    if dw_g0 is not None:
        dw_g = dw_g + _f64(dw_g0).reshape(K, N)
    if dw_fc0 is not None:
        dw_fc = dw_fc + _f64(dw_fc0).reshape(K, N)
    return dw_g, dw_fc


def x_ref(dg, dfc, w_g, w_fc):
    """x stage [SwiGLU page, formula 4]: dx = dg W_g^T + dfc W_fc^T.

    dg, dfc: [M, N]; w_g, w_fc: [K, N].  Returns dx [M, K] float64.
    """
    dg, dfc, w_g, w_fc = _f64(dg), _f64(dfc), _f64(w_g), _f64(w_fc)
    return dg @ w_g.T + dfc @ w_fc.T


def swiglu_forward_ref(x, w_g, b_g, w_fc, b_fc):
    """SwiGLU forward [SwiGLU page, operator background]:
    Gate = x W_g + b_g, FC = x W_fc + b_fc, y = SiLU(Gate) * FC.
    Returns (g, fc, y) in float64 (no rounding)."""
    x = _f64(x)
    g = x @ _f64(w_g) + _f64(b_g)
    fc = x @ _f64(w_fc) + _f64(b_fc)
    return g, fc, silu(g) * fc


def swiglu_bwd_ref(dy, x, w_g, w_fc, g, fc):
    """All seven gradients of the three-stage backward, chained in float64
    (b, then w and x consume the unrounded dg and dfc)."""
    dg, dfc, db_g, db_fc = b_ref(dy, g, fc)
    dw_g, dw_fc = w_ref(x, dg, dfc)
    dx = x_ref(dg, dfc, w_g, w_fc)
    return {"dg": dg, "dfc": dfc, "db_g": db_g, "db_fc": db_fc,
            "dw_g": dw_g, "dw_fc": dw_fc, "dx": dx}


def layer_norm_ref(x, w, b, eps):
    """y = (x - mean) / sqrt(var + eps) * w + b over the last axis; returns (y, mean, rstd).
    ``w`` / ``b`` None: 1 / 0."""
    x = _f64(x)
    mean = x.mean(1)
    d = x - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).mean(1) + eps)
    y = d * rstd[:, None]
    if w is not None:
        y = y * _f64(w)
    if b is not None:
        y = y + _f64(b)
    return y, mean, rstd


def layer_norm_bwd_ref(dy, x, w, mean, rstd):
    """Gradients (dx, dw, db) of layer_norm_ref with the statistics given."""
    dy, x = _f64(dy), _f64(x)
    rs = _f64(rstd)[:, None]
    xh = (x - _f64(mean)[:, None]) * rs
    h = dy if w is None else dy * _f64(w)
    c1 = h.mean(1, keepdims=True)
    c2 = (h * xh).mean(1, keepdims=True)
    return rs * (h - c1 - xh * c2), (dy * xh).sum(0), dy.sum(0)


def log_softmax_ref(z, t):
    """(log p, lse) of softmax(z / t) over the last axis.  z = -inf has log p = -inf; a row of
    nothing else has lse = -inf and log p = -inf."""
    a = _f64(z) / t
    m = a.max(1, keepdims=True)
    m = np.where(np.isneginf(m), 0.0, m)
    with np.errstate(divide="ignore", invalid="ignore"):
        lse = m + np.log(np.exp(a - m).sum(1, keepdims=True))
        lp = np.where(np.isneginf(a), -np.inf, a - lse)
    return lp, lse[:, 0]


def entropy_ref(lp):
    """- sum p log p, terms with p = 0 counting 0."""
    p = np.exp(lp)
    with np.errstate(invalid="ignore"):
        return -np.where(p > 0, p * lp, 0.0).sum(1)


def top_ref(z, k):
    """Ids of the k largest entries of each row: largest first, equal ones by rising index,
    NaN as -inf."""
    z = _f64(z)
    z = np.where(np.isnan(z), -np.inf, z)
    return np.argsort(-z, axis=1, kind="stable")[:, :k]


def token_logprobs_bwd_ref(z, t, targets, live, lse, entropy, g, h):
    """d(sum g logprob + h entropy)/dz with lse and entropy given; ``live`` marks the rows
    whose target counts."""
    with np.errstate(invalid="ignore"):
        lp = _f64(z) / t - _f64(lse)[:, None]
    lp = np.where(np.isneginf(_f64(z)), -np.inf, lp)
    p = np.exp(lp)
    g = np.where(live, _f64(g), 0.0)
    with np.errstate(invalid="ignore"):
        ent = np.where(p > 0, p * (lp + _f64(entropy)[:, None]), 0.0)
    d = -g[:, None] * p - _f64(h)[:, None] * ent
    rows = np.flatnonzero(live)
    d[rows, np.asarray(targets)[rows]] += g[rows]
    return d / t


def teacher_ref(u, ids, V, t):
    """(log q, q) of the teacher's entries; ids outside [0, V) are padding; a row without any
    entry above -inf has q = 0."""
    u = np.where((ids >= 0) & (ids < V), _f64(u) / t, -np.inf)
    lq, _ = log_softmax_ref(u, 1.0)
    return lq, np.exp(lq)


def distill_ref(z, t, u, ids):
    """(loss, lse): t^2 sum q (log q - log p) over the teacher's entries."""
    V = z.shape[1]
    lp, lse = log_softmax_ref(z, t)
    lq, q = teacher_ref(u, ids, V, t)
    at = np.take_along_axis(lp, np.clip(ids, 0, V - 1), 1)
    with np.errstate(invalid="ignore"):
        return t * t * np.where(q > 0, q * (lq - at), 0.0).sum(1), lse


def distill_bwd_ref(z, t, u, ids, lse, c):
    """c t (Q p - q scattered to its ids), 0 where c = 0."""
    z = _f64(z)
    V = z.shape[1]
    _, q = teacher_ref(u, ids, V, t)
    with np.errstate(invalid="ignore"):
        p = np.where(np.isneginf(z), 0.0, np.exp(z / t - _f64(lse)[:, None]))
    d = p * (q.sum(1, keepdims=True) > 0)
    for r in range(z.shape[0]):
        np.subtract.at(d[r], np.clip(ids[r], 0, V - 1), q[r])
    c = _f64(c)[:, None]
    with np.errstate(invalid="ignore"):
        return np.where(c == 0, 0.0, c * t * d)
