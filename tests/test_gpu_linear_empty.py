"""The linear layer's gradients without columns, under every activation."""
from __future__ import annotations

import pytest
import torch

import swish_activation_backward_amd as swg
from gpu_util import device, note

pytestmark = pytest.mark.gpu

ACTS = ["none", "relu", "swish", "gelu", "gelu_tanh"]


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16, torch.float32])
def test_no_columns(dt, act):
    """N = 0: dx is 0, whatever the activation."""
    note(f"linear backward N=0 {dt} {act}")
    dev = device()
    e = lambda *s: torch.empty(*s, dtype=dt, device=dev)  # noqa: E731
    for M in (5, 300):
        dx = torch.full((M, 16), 3.0, dtype=dt, device=dev)
        swg.linear_bwd(e(M, 0), e(M, 16), e(16, 0), e(M, 0), dx, e(16, 0), e(0), act)
        torch.cuda.synchronize()
        assert not dx.any()
