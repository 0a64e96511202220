"""The residual norm's backward pass of a row of more than 2^29 elements."""
from __future__ import annotations

import pytest
import torch

import swish_activation_backward_amd as swg
from gpu_util import device, note

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def test_columns_beyond_2_29():
    """One row: dw_pre = dnorm xh and, with dout alone, dw_post = D y, element by element."""
    N = (1 << 29) + 3
    note(f"residual norm M=1 N={N}")
    dev = device()
    g = torch.Generator(device="cuda").manual_seed(9)
    line = torch.randn(1 << 20, device=dev, generator=g).to(BF16)
    y = torch.cat((line.repeat(512), line[:3]))[None]
    d = torch.cat((line.flip(0).repeat(512), line[5:8]))[None]
    dwp, dwq = (torch.full((N,), float("nan"), dtype=BF16, device=dev) for _ in range(2))
    one = torch.ones(1, device=dev)
    swg.residual_norm_bwd(None, d, y, y, None, None, None, None, one, None, None, None, dwq)
    swg.residual_norm_bwd(d, None, y, None, None, None, None, one, None, None, None, dwp)
    torch.cuda.synchronize()
    for got in (dwp, dwq):                      # of statistics of 1: one product, rounded once
        for at in (0, N - (1 << 22)):
            here = slice(at, at + (1 << 22))
            assert torch.equal(got[here], (d[0, here].float() * y[0, here].float()).to(BF16))
        for at in range(0, N, 1 << 27):
            assert not got[at:at + (1 << 27)].isnan().any()
