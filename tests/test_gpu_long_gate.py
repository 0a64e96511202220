"""The b stage's column sums of more than 2^27 columns."""
from __future__ import annotations

import pytest
import torch

import swish_activation_backward_amd as swg
from gpu_util import device, note

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def test_columns_beyond_2_27():
    """One row: db is dg and dfc, which are the same fp32 values rounded once."""
    N = (1 << 27) + 24
    note(f"b stage M=1 N={N}")
    dev = device()
    g = torch.Generator(device="cuda").manual_seed(3)
    a = [torch.randn(1, N, device=dev, generator=g).to(BF16) for _ in range(3)]
    dg, dfc = torch.empty_like(a[0]), torch.empty_like(a[0])
    db_g, db_fc = torch.zeros(N, dtype=BF16, device=dev), torch.zeros(N, dtype=BF16, device=dev)
    swg.swiglu_bwd_b(*a, dg, dfc, db_g, db_fc)
    torch.cuda.synchronize()
    assert torch.equal(db_g, dg[0]) and torch.equal(db_fc, dfc[0])
    assert db_g[-24:].any() and db_fc[-24:].any()
