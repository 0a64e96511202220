"""The residual norm's statistics buffers are checked where they are given, asked for or not."""
from __future__ import annotations

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import swish_activation_backward_amd as swg


@pytest.mark.parametrize("stats", [False, True])
def test_wrong_buffers_are_refused(stats):
    with FakeTensorMode():
        f = lambda *s, dt=torch.float32: torch.empty(*s, dtype=dt, device="cuda:0")  # noqa: E731
        y = f(4, 8, dt=torch.bfloat16)
        for name in ("rstd_post", "rstd_pre"):
            for bad in (f(5), f(4, 1), f(4, dt=torch.float16), f(8)[::2],
                        torch.empty(4)):
                with pytest.raises(ValueError, match=name):
                    swg.residual_norm_fwd(y, None, stats=stats, **{name: bad})
            with pytest.raises(TypeError, match=name):
                swg.residual_norm_fwd(y, None, stats=stats, **{name: 1.0})
