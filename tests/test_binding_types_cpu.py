"""Arguments of the row operators' binding that are no tensors: TypeError, whichever they are."""
from __future__ import annotations

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import swish_activation_backward_amd as swg

NORM = ["y", "residual", "w_post", "w_pre", "gate", "out", "norm", "rstd_post", "rstd_pre"]
NORM_BWD = ["dout", "dnorm", "y", "out", "w_post", "w_pre", "gate", "rstd_post", "rstd_pre", "dy",
            "dresidual", "dw_post", "dw_pre", "dgate"]
LINEAR = ["x", "w", "bias", "residual", "y", "z"]
LINEAR_BWD = ["dy", "x", "w", "z", "dx", "dw", "db"]
LAYER = ["x", "w", "b", "y", "mean", "rstd"]


def refuses(call, args, names, keep=()):
    for n in names:
        with pytest.raises(TypeError, match=f"{n} must be"):
            call(**{**{k: v for k, v in args.items() if k not in keep}, n: 3.0})


def test_what_is_no_tensor_is_refused():
    with FakeTensorMode():
        f = lambda *s: torch.empty(*s, dtype=torch.float32, device="cuda:0")  # noqa: E731
        m, v, r = f(4, 8), f(8), f(4)
        refuses(swg.residual_norm_fwd, dict(y=m, residual=m, w_post=v, w_pre=v, gate=v), NORM)
        # alone: nothing else says a type
        refuses(swg.residual_norm_fwd, dict(y=m, residual=None), NORM)
        a = dict(dout=m, dnorm=m, y=m, out=m, w_post=v, w_pre=v, gate=v, rstd_post=r, rstd_pre=r,
                 dy=m, dresidual=m, dw_post=v, dw_pre=v, dgate=v)
        refuses(swg.residual_norm_bwd, a, NORM_BWD)
        a = dict(x=f(4, 6), w=f(6, 8), bias=v, residual=m)
        refuses(swg.linear_fwd, a, LINEAR)
        a = dict(dy=m, x=f(4, 6), w=f(6, 8), z=m, dx=f(4, 6), dw=f(6, 8), db=v, act="gelu")
        refuses(swg.linear_bwd, a, LINEAR_BWD)
        refuses(swg.layer_norm_fwd, dict(x=m, w=v, b=v), LAYER)
        refuses(swg.layer_norm_fwd, dict(x=m, w=None, b=None), LAYER)
