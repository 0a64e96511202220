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

Around the gate, in the same manner: ``layer_norm`` / ``LayerNorm``, ``token_logprobs`` (log
probability of given tokens and entropy) and ``distill_loss`` (a teacher's top logits).
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
    x2 = x.reshape(-1, x.shape[-1])
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
