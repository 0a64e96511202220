"""Drop-in training use: a ``torch.autograd.Function`` and an ``nn.Module`` for the SwiGLU
feed-forward gate whose forward and backward both run in the library's kernels.

    y = SiLU(x W_g + b_g) * (x W_fc + b_fc)

Forward: ``swiglu_fwd`` (g, fc and y from one fused GEMM); g and fc are saved for the
backward, which runs the three stages of the Fused SwiGLU backward page's call chain
(b -> w -> x): ``swiglu_bwd_b`` (dg, dfc, db), then, when both dW and dx are needed, the
fused ``swiglu_bwd_wx`` (both GEMMs over [dg | dfc] from one launch in bf16 / fp16),
otherwise ``swiglu_bwd_w`` (dW) or ``swiglu_bwd_x`` (dx).  The pattern is a custom operator whose backward hook calls a hand-written gradient
kernel (the Ascend C custom-backward page, "突破自动微分瓶颈: 基于 Ascend C 的高性能自定义反向传播
算子实战", section 4.2, Python-side registration); the weight layout [K, N] is the SwiGLU
page's.  Leading dimensions of x are flattened into M.

Around the gate, in the same manner: ``layer_norm`` / ``LayerNorm``, ``linear`` / ``Linear`` (with
bias, activation and residual), ``residual_norm`` (the norms around a block with its gate and the
residual sum), ``token_logprobs`` (log probability of given tokens and entropy) and ``distill_loss``
(a teacher's top logits).  ``Block`` puts a gated feed-forward together from them.
"""
from __future__ import annotations

import math

import torch
from torch.autograd.function import once_differentiable

from . import _lib


class SwiGLUFunction(torch.autograd.Function):
    """x [M, K], w_g / w_fc [K, N], b_g / b_fc [N] or None -> y [M, N] (bf16, fp16 or fp32,
    contiguous, on the GPU)."""

    @staticmethod
    def forward(ctx, x, w_g, w_fc, b_g, b_fc):
        M, N = x.shape[0], w_g.shape[1]
        g = torch.empty(M, N, dtype=x.dtype, device=x.device)
        fc = torch.empty_like(g)
        y = torch.empty_like(g)
        _lib.swiglu_fwd(x, w_g, w_fc, b_g, b_fc, g, fc, y)
        ctx.save_for_backward(x, w_g, w_fc, g, fc)
        ctx.has_bias = (b_g is not None, b_fc is not None)
        return y

    @staticmethod
    def backward(ctx, dy):
        x, w_g, w_fc, g, fc = ctx.saved_tensors
        dy = dy.contiguous()
        M, N = g.shape
        K = x.shape[1]
        dg, dfc = torch.empty_like(g), torch.empty_like(fc)
        db_g = torch.zeros(N, dtype=g.dtype, device=g.device)
        db_fc = torch.zeros_like(db_g)
        _lib.swiglu_bwd_b(dy, g, fc, dg, dfc, db_g, db_fc)
        dx = dw_g = dw_fc = None
        need_w = ctx.needs_input_grad[1] or ctx.needs_input_grad[2]
        if need_w and ctx.needs_input_grad[0]:
            dw_g = torch.zeros(K, N, dtype=g.dtype, device=g.device)
            dw_fc = torch.zeros_like(dw_g)
            dx = torch.empty(M, K, dtype=x.dtype, device=x.device)
            _lib.swiglu_bwd_wx(x, dg, dfc, w_g, w_fc, dw_g, dw_fc, dx)
            return (dx, dw_g, dw_fc, db_g if ctx.has_bias[0] else None,
                    db_fc if ctx.has_bias[1] else None)
        if need_w:
            dw_g = torch.zeros(K, N, dtype=g.dtype, device=g.device)
            dw_fc = torch.zeros_like(dw_g)
            _lib.swiglu_bwd_w(x, dg, dfc, dw_g, dw_fc)
        if ctx.needs_input_grad[0]:
            dx = torch.empty(M, K, dtype=x.dtype, device=x.device)
            _lib.swiglu_bwd_x(dg, dfc, w_g, w_fc, dx)
        return (dx, dw_g, dw_fc, db_g if ctx.has_bias[0] else None,
                db_fc if ctx.has_bias[1] else None)


def swiglu(x, w_g, w_fc, b_g=None, b_fc=None):
    """SwiGLU gate over the last dimension of x (any leading shape)."""
    lead = x.shape[:-1]
    x2 = x.reshape(-1, x.shape[-1]).contiguous()
    y = SwiGLUFunction.apply(x2, w_g, w_fc, b_g, b_fc)
    return y.view(*lead, w_g.shape[1])


class SwiGLU(torch.nn.Module):
    """Parameters w_g, w_fc [in_features, hidden] and optional biases [hidden]; forward(x)
    maps [..., in_features] to [..., hidden]."""

    def __init__(self, in_features, hidden, bias=True, device=None, dtype=torch.bfloat16):
        super().__init__()
        kw = {"device": device, "dtype": dtype}
        self.w_g = torch.nn.Parameter(torch.empty(in_features, hidden, **kw))
        self.w_fc = torch.nn.Parameter(torch.empty(in_features, hidden, **kw))
        if bias:
            self.b_g = torch.nn.Parameter(torch.zeros(hidden, **kw))
            self.b_fc = torch.nn.Parameter(torch.zeros(hidden, **kw))
        else:
            self.register_parameter("b_g", None)
            self.register_parameter("b_fc", None)
        bound = 1.0 / math.sqrt(in_features)
        with torch.no_grad():
            self.w_g.uniform_(-bound, bound)
            self.w_fc.uniform_(-bound, bound)

    def forward(self, x):
        return swiglu(x, self.w_g, self.w_fc, self.b_g, self.b_fc)


def _rows_of(x):
    """x [..., N] as a matrix of contiguous rows (a view where its layout allows)."""
    x2 = x.reshape(math.prod(x.shape[:-1]), x.shape[-1])
    R, C = x2.shape
    if (C > 1 and x2.stride(1) != 1) or (R > 1 and x2.stride(0) < C):
        x2 = x2.contiguous()
    return x2


class LayerNormFunction(torch.autograd.Function):
    """x [M, N], w / b [N] or None -> y [M, N]."""

    @staticmethod
    def forward(ctx, x, w, b, eps):
        y, mean, rstd = _lib.layer_norm_fwd(x, w, b, eps=eps)
        ctx.save_for_backward(x, w, mean, rstd)
        ctx.wdtype = next((t.dtype for t in (w, b) if t is not None), x.dtype)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, w, mean, rstd = ctx.saved_tensors
        dy = _rows_of(dy)
        need_x, need_w, need_b = ctx.needs_input_grad[:3]
        N, dev = x.shape[1], x.device
        dx = torch.empty(x.shape, dtype=x.dtype, device=dev) if need_x else None
        dw = torch.empty(N, dtype=ctx.wdtype, device=dev) if need_w else None
        db = torch.empty(N, dtype=ctx.wdtype, device=dev) if need_b else None
        _lib.layer_norm_bwd(dy, x, w, mean, rstd, dx, dw, db)
        return dx, dw, db, None


def layer_norm(x, w=None, b=None, eps=1e-5):
    """Layer norm over the last dimension of x (any leading shape); ``w`` and ``b`` have x's
    dtype or fp32."""
    return LayerNormFunction.apply(_rows_of(x), w, b, eps).view(x.shape)


class LayerNorm(torch.nn.Module):
    """Parameters w (ones) and b (zeros, optional) [features], of ``dtype`` (fp32 goes with any
    activations); forward(x) norms [..., features]."""

    def __init__(self, features, eps=1e-5, bias=True, device=None, dtype=torch.float32):
        super().__init__()
        self.eps = eps
        self.w = torch.nn.Parameter(torch.ones(features, device=device, dtype=dtype))
        if bias:
            self.b = torch.nn.Parameter(torch.zeros(features, device=device, dtype=dtype))
        else:
            self.register_parameter("b", None)

    def forward(self, x):
        return layer_norm(x, self.w, self.b, self.eps)


class LinearFunction(torch.autograd.Function):
    """x [M, K], w [K, N] (or the transpose of a [N, K]), b [N] or None, residual [M, N] or None
    -> y [M, N]."""

    @staticmethod
    def forward(ctx, x, w, b, residual, act, beta):
        M, N = x.shape[0], w.shape[1]
        z = None
        if act != "none" and any(ctx.needs_input_grad[:3]):
            z = torch.empty(M, N, dtype=x.dtype, device=x.device)
        y = _lib.linear_fwd(x, w, b, residual, act, beta, z=z)
        ctx.save_for_backward(x, w, z)
        ctx.act, ctx.beta = act, beta
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, w, z = ctx.saved_tensors
        dy = _rows_of(dy)
        need_x, need_w, need_b, need_r = ctx.needs_input_grad[:4]
        (M, K), N, dev = x.shape, w.shape[1], x.device
        dx = torch.empty(M, K, dtype=x.dtype, device=dev) if need_x else None
        dw = None
        if need_w:   # stored as w is
            rows = N <= 1 or w.stride(1) == 1
            dw = torch.empty((K, N) if rows else (N, K), dtype=x.dtype, device=dev)
            dw = dw if rows else dw.t()
        db = torch.empty(N, dtype=x.dtype, device=dev) if need_b else None
        if need_x or need_w or need_b:
            _lib.linear_bwd(dy, x if need_w else None, w if need_x else None, z, dx, dw, db,
                            ctx.act, ctx.beta)
        return dx, dw, db, dy if need_r else None, None, None


def linear(x, w, b=None, residual=None, act="none", beta=1.0):
    """act(x w + b) + residual over the last dimension of x (any leading shape), w [K, N] or the
    transpose of a [N, K], residual [..., N].  ``act``: "none", "relu", "swish" (z sigma(beta z)),
    "gelu" or "gelu_tanh"."""
    if residual is not None:
        residual = _rows_of(residual)
    y = LinearFunction.apply(_rows_of(x), w, b, residual, act, beta)
    return y.view(*x.shape[:-1], w.shape[1])


class Linear(torch.nn.Module):
    """Parameters w [in_features, out_features] and b (optional); forward(x, residual) is
    act(x w + b) + residual."""

    def __init__(self, in_features, out_features, bias=True, act="none", beta=1.0, device=None,
                 dtype=torch.bfloat16):
        super().__init__()
        kw = {"device": device, "dtype": dtype}
        self.act, self.beta = act, beta
        self.w = torch.nn.Parameter(torch.empty(in_features, out_features, **kw))
        if bias:
            self.b = torch.nn.Parameter(torch.zeros(out_features, **kw))
        else:
            self.register_parameter("b", None)
        bound = 1.0 / math.sqrt(in_features)
        with torch.no_grad():
            self.w.uniform_(-bound, bound)

    def forward(self, x, residual=None):
        return linear(x, self.w, self.b, residual, self.act, self.beta)


class ResidualNormFunction(torch.autograd.Function):
    """y [M, N], residual [M, N] or None, w_post, w_pre [N] or None, gate [N], [M, 1], [M, N] or
    None -> out [M, N], norm [M, N] (None where ``pre`` is off)."""

    @staticmethod
    def forward(ctx, y, residual, w_post, w_pre, gate, scale, eps, post, pre):
        r = _lib.residual_norm_fwd(y, residual, w_post, w_pre, gate, scale, post, pre, eps=eps,
                                   stats=True)
        ctx.save_for_backward(y, r.out, w_post, w_pre, gate, r.rstd_post, r.rstd_pre)
        ctx.scale = scale
        ctx.set_materialize_grads(False)
        return r.out, r.norm

    @staticmethod
    @once_differentiable
    def backward(ctx, dout, dnorm):
        none = (None,) * 4
        if dout is None and dnorm is None:
            return (None,) * 5 + none
        y, out, w_post, w_pre, gate, rstd_post, rstd_pre = ctx.saved_tensors
        need_y, need_r, need_wp, need_wq, need_g = ctx.needs_input_grad[:5]
        new = lambda t, like, need: (torch.empty(like.shape, dtype=t.dtype,  # noqa: E731
                                                 device=t.device) if need else None)
        dy, dr = new(y, y, need_y), new(out, out, need_r)
        # a weight of a norm that is off has no part in the result
        dwp = new(w_post, w_post, True) if need_wp and rstd_post is not None else None
        dwq = new(w_pre, w_pre, True) if need_wq and rstd_pre is not None else None
        dg = new(gate, gate, True) if need_g else None
        _lib.residual_norm_bwd(None if dout is None else _rows_of(dout),
                               None if dnorm is None else _rows_of(dnorm), y, out, w_post, w_pre,
                               gate, rstd_post, rstd_pre, dy, dr, dwp, dwq, dg, scale=ctx.scale)
        return (dy, dr, dwp, dwq, dg) + none


def residual_norm(y, residual=None, w_post=None, w_pre=None, gate=None, scale=1.0, eps=1e-5,
                  post=True, pre=True):
    """The root mean square norm after a block (``post``), its gate, the residual sum and the norm
    before the next block (``pre``) over the last dimension of y (any leading shape): returns

        out = residual + scale * gate * rms(y) w_post  and  norm = rms(out) w_pre

    (norm None without ``pre``).  ``gate`` is None, [N], or of y's leading shape with 1 or N
    elements a row."""
    if residual is not None:
        residual = _rows_of(residual)
    if gate is not None and gate.dim() != 1:
        gate = gate.reshape(-1, 1) if gate.shape[-1] == 1 else _rows_of(gate)
    out, norm = ResidualNormFunction.apply(_rows_of(y), residual, w_post, w_pre, gate, scale, eps,
                                           post, pre)
    return out.view(y.shape), None if norm is None else norm.view(y.shape)


class Block(torch.nn.Module):
    """A gated feed-forward between two norms: forward(stream, normed) returns the next stream and
    the norm that the next block takes,

        y = linear(swiglu(normed)),  stream + scale * gate * rms(y) w_post,  rms(that) w_pre

    The norms' weights and the gate (one value a channel) are fp32.  The stream is of ``dtype`` or
    fp32, ``normed`` of ``dtype``; ``enter`` norms a stream for the first block."""

    def __init__(self, features, hidden, scale=1.0, eps=1e-5, bias=True, device=None,
                 dtype=torch.bfloat16):
        super().__init__()
        self.scale, self.eps = scale, eps
        self.swiglu = SwiGLU(features, hidden, bias, device, dtype)
        self.out = Linear(hidden, features, bias, device=device, dtype=dtype)
        ones = lambda: torch.nn.Parameter(torch.ones(features, device=device))  # noqa: E731
        self.w_post, self.w_pre, self.gate = ones(), ones(), ones()

    @staticmethod
    def enter(stream, w=None, eps=1e-5):
        """The norm in front of the first block, of the stream's dtype: an fp32 stream over 16-bit
        blocks is cast before (``Block.enter(stream.to(dtype))``) or its norm after."""
        return residual_norm(stream, None, None, w, eps=eps, post=False)[1]

    def forward(self, stream, normed):
        y = self.out(self.swiglu(normed))
        return residual_norm(y, stream, self.w_post, self.w_pre, self.gate, self.scale, self.eps)


class TokenLogprobsFunction(torch.autograd.Function):
    """logits [R, V], targets [R] (int64) -> logprob [R], entropy [R] (fp32)."""

    @staticmethod
    def forward(ctx, logits, targets, temperature, ignore_index):
        r = _lib.token_logprobs(logits, targets, temperature=temperature,
                                ignore_index=ignore_index)
        ctx.save_for_backward(logits, targets, r.lse, r.entropy)
        ctx.temperature, ctx.ignore_index = temperature, ignore_index
        ctx.set_materialize_grads(False)
        return r.logprob, r.entropy

    @staticmethod
    @once_differentiable
    def backward(ctx, dlogprob, dentropy):
        if not ctx.needs_input_grad[0] or (dlogprob is None and dentropy is None):
            return None, None, None, None
        logits, targets, lse, entropy = ctx.saved_tensors
        dlogits = _lib.token_logprobs_bwd(
            logits, None if dlogprob is None else targets, lse,
            None if dentropy is None else entropy,
            None if dlogprob is None else dlogprob.contiguous(),
            None if dentropy is None else dentropy.contiguous(),
            torch.empty(logits.shape, dtype=logits.dtype, device=logits.device),
            temperature=ctx.temperature, ignore_index=ctx.ignore_index)
        return dlogits, None, None, None


def token_logprobs(logits, targets, temperature=1.0, ignore_index=-100):
    """Log probability of each of the ``targets`` [...] (int64) under
    softmax(logits / temperature), logits [..., V], and the entropy, both fp32 of shape [...]
    and differentiable with respect to the logits."""
    lp, ent = TokenLogprobsFunction.apply(_rows_of(logits), targets.reshape(-1).contiguous(),
                                          temperature, ignore_index)
    return lp.view(targets.shape), ent.view(targets.shape)


class DistillFunction(torch.autograd.Function):
    """logits [R, V], top and top_ids [R, k] -> loss [R] (fp32)."""

    @staticmethod
    def forward(ctx, logits, top, top_ids, temperature):
        loss, lse = _lib.distill_fwd(logits, top, top_ids, temperature=temperature)
        ctx.save_for_backward(logits, top, top_ids, lse)
        ctx.temperature = temperature
        return loss

    @staticmethod
    @once_differentiable
    def backward(ctx, dloss):
        if not ctx.needs_input_grad[0]:
            return None, None, None, None
        logits, top, top_ids, lse = ctx.saved_tensors
        dlogits = _lib.distill_bwd(
            logits, top, top_ids, lse, dloss.contiguous(),
            torch.empty(logits.shape, dtype=logits.dtype, device=logits.device),
            temperature=ctx.temperature)
        return dlogits, None, None, None


def distill_loss(logits, top, top_ids, temperature=1.0):
    """Distillation loss [...] (fp32) of logits [..., V] against a teacher's entries ``top``
    and ``top_ids`` [..., k], e.g. what ``token_logprobs`` of the binding returned for the
    teacher's logits; differentiable with respect to the logits (the teacher's entries are
    constants).  ``distill_fwd_bwd`` of the binding forms the same loss with its gradient in
    one pass where the row weights are known beforehand."""
    k = top.shape[-1]
    loss = DistillFunction.apply(_rows_of(logits), top.detach().reshape(-1, k).contiguous(),
                                 top_ids.reshape(-1, k).contiguous(), temperature)
    return loss.view(logits.shape[:-1])
