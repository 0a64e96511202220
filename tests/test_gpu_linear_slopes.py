"""Slopes of the linear layer's activations at pre-activations that their type holds as an infinity
or as its largest value."""
from __future__ import annotations

import pytest
import torch

import swish_activation_backward_amd as swg
from gpu_util import device, note

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
# activation, beta, slope for large positive z, for large negative z
LIMITS = [("relu", 1.0, 1.0, 0.0), ("swish", 1.0, 1.0, 0.0), ("swish", 1.7, 1.0, 0.0),
          ("swish", -2.0, 0.0, 1.0), ("swish", 0.0, 0.5, 0.5), ("swish", 1e38, 1.0, 0.0),
          ("gelu", 1.0, 1.0, 0.0), ("gelu_tanh", 1.0, 1.0, 0.0)]


@pytest.mark.parametrize("N", [5, 40, 523])
@pytest.mark.parametrize("act,beta,up,down", LIMITS)
@pytest.mark.parametrize("dt", [BF16, FP16, FP32])
def test_slopes_of_large_pre_activations(dt, act, beta, up, down, N):
    note(f"linear slopes {dt} {act} {beta} N={N}")
    dev = device()
    most = torch.finfo(dt).max
    z = torch.tensor([float("inf"), -float("inf"), most, -most, float("nan")], dtype=dt, device=dev)
    want = torch.tensor([up, down, up, down, float("nan")], dtype=dt, device=dev)
    rep = -(-N // 5)
    z, want = z.repeat(rep)[None, :N].contiguous(), want.repeat(rep)[:N]
    dy, x = torch.full_like(z, 2.0), torch.ones(1, 1, dtype=dt, device=dev)
    dw, db = torch.empty(1, N, dtype=dt, device=dev), torch.empty(N, dtype=dt, device=dev)
    swg.linear_bwd(dy, x, None, z, None, dw, db, act, beta)
    torch.cuda.synchronize()
    for got in (dw[0], db):
        assert torch.equal(got.isnan(), want.isnan())
        assert torch.equal(got.nan_to_num(), 2 * want.nan_to_num())


@pytest.mark.parametrize("act", ["relu", "swish", "gelu", "gelu_tanh"])
def test_a_finite_forward_has_finite_gradients(act):
    """fp16 pre-activations of -90000 are kept as -inf: their outputs are 0, and so are their
    gradients."""
    dev = device()
    x = torch.full((9, 3), 300.0, dtype=FP16, device=dev)
    w = torch.full((3, 16), -100.0, dtype=FP16, device=dev)
    z = torch.empty(9, 16, dtype=FP16, device=dev)
    y = swg.linear_fwd(x, w, act=act, z=z)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty(16, dtype=FP16, device=dev)
    swg.linear_bwd(torch.ones_like(y), x, w, z, dx, dw, db, act)
    torch.cuda.synchronize()
    assert (z == -float("inf")).all() and not y.any()
    assert not dx.any() and not dw.any() and not db.any()
