"""The residual norm's statistics: written where a buffer is given or they are asked for."""
from __future__ import annotations

import pytest
import torch

import swish_activation_backward_amd as swg
from gpu_util import device

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("stats", [False, True])
@pytest.mark.parametrize("given", ["post", "pre", "both"])
@pytest.mark.parametrize("N", [5, 64, 4096, 20000])
def test_given_buffers_are_written(N, given, stats):
    dev = device()
    g = torch.Generator().manual_seed(N)
    y, res = (torch.randn(7, N, generator=g).to(dev) for _ in range(2))
    want = swg.residual_norm_fwd(y, res, stats=True)
    a, b = (torch.full((7,), float("nan"), device=dev) for _ in range(2))
    r = swg.residual_norm_fwd(y, res, stats=stats, rstd_post=a if given != "pre" else None,
                              rstd_pre=b if given != "post" else None)
    torch.cuda.synchronize()
    for got, buf, ref, here in ((r.rstd_post, a, want.rstd_post, given != "pre"),
                                (r.rstd_pre, b, want.rstd_pre, given != "post")):
        assert (got is buf) == here
        if here or stats:
            assert torch.equal(got, ref)
        else:
            assert got is None


def test_buffers_of_a_norm_that_is_off_stay():
    dev = device()
    y = torch.randn(7, 64, device=dev)
    a, b = (torch.full((7,), 3.0, device=dev) for _ in range(2))
    r = swg.residual_norm_fwd(y, None, post=False, rstd_post=a, rstd_pre=b)
    q = swg.residual_norm_fwd(y, None, pre=False, rstd_post=b.clone(), rstd_pre=a)
    torch.cuda.synchronize()
    assert (a == 3).all() and r.rstd_post is None and q.rstd_pre is None
    assert r.rstd_pre is b and not (b == 3).any() and not (q.rstd_post == 3).any()
