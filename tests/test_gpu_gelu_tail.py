"""gelu of the linear layer below 0, relative to itself."""
from __future__ import annotations

import numpy as np
import pytest
import torch
from scipy.special import erfc

import swish_activation_backward_amd as swg
from gpu_util import device
from parity import to64

pytestmark = pytest.mark.gpu


def test_gelu_tail():
    """In units of u = 2^-24: the exponent z^2 / 2 is a product of
    three factors, one of them a rounded constant, which moves the exponential by at most
    2.5 z^2 / 2; the exponential 2; t = 1 / (1 + 0.3 x) 4 units, times at most 3.8 for what t p(t)
    makes of them; its coefficients and the steps of its evaluation 5, the fit 0.7, the products and
    the output's rounding 4: 32 at most."""
    dev = device()
    z = torch.linspace(-12.5, 0.0, 200001, device=dev)[:, None].contiguous()
    y = swg.linear_fwd(z, torch.ones(1, 1, device=dev), act="gelu")
    torch.cuda.synchronize()
    z64 = to64(z)[:, 0]
    want = 0.5 * z64 * erfc(-z64 / np.sqrt(2.0))
    err = np.abs(to64(y)[:, 0] - want)
    assert (err <= 2.0 ** -24 * (32 + 1.25 * z64 * z64) * np.abs(want)).all()
