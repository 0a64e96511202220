"""Rows whose values lie far from zero beside what they differ by: the mean is the rounded quotient
of the sum by N."""
from __future__ import annotations

import pytest
import torch

import swish_activation_backward_amd as swg
from gpu_util import device, note

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
# every kernel's range of row lengths, odd ones among them
WIDTHS = [1, 5, 8, 9, 56, 100, 127, 250, 511, 513, 1000, 1023, 2000, 3001, 4095, 5000, 8191, 12345,
          16383, 20001]


def equal_values(dt):
    """Values of 8 significant bits: their multiples by up to 2^16 are fp32 numbers, and every
    order of adding them up is exact."""
    if dt == FP16:
        return [3.0, 1020.0, 60160.0, -65024.0]
    return [3.0, 1020.0, 99840.0, -9961472.0, 2.0 ** 66]


@pytest.mark.parametrize("dt", [BF16, FP16, FP32])
@pytest.mark.parametrize("N", WIDTHS)
def test_rows_of_equal_values(N, dt):
    """mean is the value itself, so y = b and rstd = 1 / sqrt(eps), whatever the value."""
    note(f"equal norm rows N={N} {dt}")
    values = torch.tensor(equal_values(dt), device=device()).to(dt)
    x = values[:, None].repeat(3, N).contiguous()
    g = torch.Generator().manual_seed(N)
    w, b = (torch.randn(N, generator=g).to(dt).to(x.device) for _ in range(2))
    y, mean, rstd = swg.layer_norm_fwd(x, w, b)
    assert torch.equal(mean, x[:, 0].float())
    assert torch.equal(y, b[None].expand_as(y))
    want = torch.full_like(rstd, 1e-5).rsqrt()
    assert bool(((rstd - want).abs() <= 2.0 ** -21 * want).all())
