"""Logits far from the ordinary range."""
from __future__ import annotations

import pytest
import torch

import swish_activation_backward_amd as swg
from gpu_util import device, note
from logit_range_models import check_forward, check_loss
from test_gpu_vocab import BF16, FP32, teacher

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ rows of large equal values
@pytest.mark.parametrize("dt", [BF16, FP32])
@pytest.mark.parametrize("value", [1e5, 1e6, 1e7, 1e8, -1e5, -1e6, -1e7, -1e8])
def test_rows_of_large_equal_values(value, dt):
    """log p = -log V whatever the value and wherever the row starts: single elements at a row's
    ends and its chunks have one reference."""
    note(f"equal values {value} {dt}")
    for V in (1, 2, 7, 14, 23, 300, 4099, 9001):
        buf = torch.full((3 * V + 8,), value, dtype=dt, device=device())
        for shift in range(8):
            z = buf[shift:shift + 3 * V].view(3, V)
            t = torch.tensor([0, V // 2, V - 1], device=z.device)
            r = swg.token_logprobs(z, t, top=min(V, 5))
            check_forward(z, t, r, 1.0, min(V, 5))
            u, ids = teacher(3, V, 2, pads=False)
            loss, lse = swg.distill_fwd(z, u, ids)
            check_loss(z, u, ids, 1.0, loss, lse)
            c = torch.ones(3, device=z.device)
            loss, lse, dz = swg.distill_fwd_bwd(z, u, ids, c)
            check_loss(z, u, ids, 1.0, loss, lse, c, dz)
