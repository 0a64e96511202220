"""The autograd wrapper of the linear layer without columns or without features."""
from __future__ import annotations

import pytest
import torch

from gpu_util import device
from swish_activation_backward_amd.autograd import linear

pytestmark = pytest.mark.gpu

ACTS = ["none", "relu", "swish", "gelu", "gelu_tanh"]


@pytest.mark.parametrize("act", ACTS)
def test_no_columns_or_no_features_through_autograd(act):
    dev = device()
    x = torch.randn(2, 5, 16, device=dev, requires_grad=True)
    w = torch.empty(16, 0, device=dev, requires_grad=True)
    y = linear(x, w, act=act)
    assert y.shape == (2, 5, 0)
    y.sum().backward()
    assert x.grad.shape == x.shape and not x.grad.any() and w.grad.shape == (16, 0)
    x = torch.empty(2, 5, 0, device=dev, requires_grad=True)
    w = torch.empty(0, 24, device=dev, requires_grad=True)
    b = torch.randn(24, device=dev, requires_grad=True)
    y = linear(x, w, b, act=act)
    assert torch.equal(y[0, 0], y[1, 4]) and (act != "none" or torch.equal(y[0, 0], b))
    y.sum().backward()
    assert x.grad.shape == x.shape and w.grad.shape == (0, 24) and b.grad.shape == (24,)
