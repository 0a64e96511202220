"""Layer norm's backward pass of a row of more than 2^29 elements."""
from __future__ import annotations

import pytest
import torch

import swish_activation_backward_amd as swg
from gpu_util import device, note

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def test_columns_beyond_2_29():
    """One row of statistics 0 and 1: dw = dy x and db = dy, element by element."""
    N = (1 << 29) + 3
    note(f"layer norm M=1 N={N}")
    dev = device()
    g = torch.Generator(device="cuda").manual_seed(9)
    line = torch.randn(1 << 20, device=dev, generator=g).to(BF16)
    x = torch.cat((line.repeat(512), line[:3]))[None]
    dy = torch.cat((line.flip(0).repeat(512), line[5:8]))[None]
    dw, db = (torch.full((N,), float("nan"), dtype=BF16, device=dev) for _ in range(2))
    swg.layer_norm_bwd(dy, x, None, torch.zeros(1, device=dev), torch.ones(1, device=dev), None, dw,
                       db)
    torch.cuda.synchronize()
    for at in (0, N - (1 << 22)):
        here = slice(at, at + (1 << 22))
        assert torch.equal(dw[here], (dy[0, here].float() * x[0, here].float()).to(BF16))
    for at in range(0, N, 1 << 27):
        here = slice(at, at + (1 << 27))
        assert torch.equal(db[here], dy[0, here]) and not dw[here].isnan().any()
