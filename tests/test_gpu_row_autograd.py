"""The autograd wrappers of layer norm, token log probabilities and distillation, and the
example that trains with them."""
from __future__ import annotations

import math

import pytest
import torch

import swish_activation_backward_amd as swg
from gpu_util import device, note
from swish_activation_backward_amd.autograd import (LayerNorm, distill_loss, layer_norm,
                                                    token_logprobs)
from workloads import distill

pytestmark = pytest.mark.gpu


def close(name, got, want, tol):
    """Normwise, the reference in float64."""
    err = (got.double() - want).norm() / want.norm().clamp_min(1e-300)
    assert err <= tol, f"{name}: {err:.3g} > {tol:.3g}"


@pytest.mark.parametrize("layout", ["dense", "leading", "transposed"])
def test_layer_norm(layout):
    dev = device()
    g = torch.Generator().manual_seed(1)
    shape = {"dense": (37, 96), "leading": (3, 5, 96), "transposed": (96, 37)}[layout]
    x = torch.randn(shape, generator=g).to(dev)
    x = (x.t() if layout == "transposed" else x).requires_grad_()
    ln = LayerNorm(96, device=dev)
    with torch.no_grad():
        ln.w.add_(torch.randn(96, generator=g).to(dev) * 0.2)
        ln.b.add_(torch.randn(96, generator=g).to(dev) * 0.2)
    y = ln(x)
    dy = torch.randn(y.shape, generator=g).to(dev)
    gx, gw, gb = torch.autograd.grad(y, (x, ln.w, ln.b), dy)
    xd, wd, bd = (t.detach().double().requires_grad_() for t in (x, ln.w, ln.b))
    yd = torch.nn.functional.layer_norm(xd, (96,), wd, bd, 1e-5)
    want = torch.autograd.grad(yd, (xd, wd, bd), dy.double())
    # rows of 96: a hundred fp32 roundings at most
    for n, a, b in zip(("y", "dx", "dw", "db"), (y, gx, gw, gb), (yd, *want)):
        assert a.shape == b.shape
        close(n, a.detach(), b.detach(), 96 * 2.0 ** -24)


def test_layer_norm_partial_gradients():
    """Frozen parameters, no parameters, and a gradient that is broadcast."""
    dev = device()
    x = torch.randn(9, 64, device=dev, requires_grad=True)
    w = torch.ones(64, device=dev, requires_grad=True)
    for ww in (w, w.detach(), None):
        y = layer_norm(x, ww)
        y.sum().backward()          # an expanded gradient
        # the gradient of a sum of normed values is 0: what is left are roundings of terms of
        # the size of rstd (1 here), 64 of them
        assert x.grad.abs().max() <= 64 * 2.0 ** -20
        x.grad = None
    assert w.grad is not None


def test_token_logprobs():
    dev = device()
    g = torch.Generator().manual_seed(2)
    z = (torch.randn(4, 7, 333, generator=g) * 2).to(dev).requires_grad_()
    t = torch.randint(0, 333, (4, 7), generator=g).to(dev)
    t[1, 2] = -100
    zd = z.detach().double().requires_grad_()
    lpd = torch.log_softmax(zd / 0.7, -1)
    td = lpd.gather(-1, t.clamp_min(0)[..., None])[..., 0] * (t != -100)
    ed = torch.special.entr(lpd.exp()).sum(-1)
    wl, we = torch.randn(2, 4, 7, generator=g).to(dev)
    for use_l, use_e in ((1, 1), (1, 0), (0, 1)):
        lp, ent = token_logprobs(z, t, temperature=0.7)
        assert lp.shape == t.shape
        close("logprob", lp.detach(), td.detach(), 400 * 2.0 ** -24)
        close("entropy", ent.detach(), ed.detach(), 400 * 2.0 ** -24)
        loss = (use_l * (wl * lp).sum() if use_l else 0) + (use_e * (we * ent).sum() if use_e else 0)
        (got,) = torch.autograd.grad(loss, z)
        ref = use_l * (wl.double() * td).sum() + use_e * (we.double() * ed).sum()
        (want,) = torch.autograd.grad(ref, zd, retain_graph=True)
        close("dlogits", got, want, 800 * 2.0 ** -24)


def test_distill_loss():
    dev = device()
    g = torch.Generator().manual_seed(3)
    z = (torch.randn(2, 5, 200, generator=g) * 2).to(dev).requires_grad_()
    teacher = torch.randn(10, 200, generator=g).to(dev) * 3
    kept = swg.token_logprobs(teacher, top=16)
    u, ids = kept.top_logprob.view(2, 5, 16), kept.top_id.view(2, 5, 16)
    loss = distill_loss(z, u, ids, 2.0)
    (got,) = torch.autograd.grad(loss.mean(), z)
    zd = z.detach().double().requires_grad_()
    q = torch.softmax(u.double() / 2, -1)
    lp = torch.log_softmax(zd / 2, -1).gather(-1, ids)
    want = 4 * (torch.special.xlogy(q, q) - q * lp).sum(-1)
    close("loss", loss.detach(), want.detach(), 400 * 2.0 ** -24)
    (gw,) = torch.autograd.grad(want.mean(), zd)
    close("dlogits", got, gw, 800 * 2.0 ** -24)


def test_example():
    note("distillation example")
    losses, before, after = distill.run(steps=12, tokens=256, width=128, hidden=256, vocab=3001)
    assert all(math.isfinite(x) for x in losses)
    assert losses[-1] < 0.7 * losses[0] and after > before


def test_one_pass_step_matches_autograd():
    dev = device()
    torch.manual_seed(4)
    student = distill.Head(64, 128, 1000, dev, torch.bfloat16)
    x = torch.randn(300, 64, device=dev, dtype=torch.bfloat16)
    kept = swg.token_logprobs(torch.randn(300, 1000, device=dev) * 3, top=8)
    distill_loss(student(x), kept.top_logprob, kept.top_id, 2.0).mean().backward()
    want = [p.grad.clone() for p in student.parameters()]
    for p in student.parameters():
        p.grad = None
    distill.train_step_in_one_pass(student, x, kept, 2.0)
    # the logit gradients differ by a rounding to bf16 here and there, and so do the sums of 300
    # rows' products behind them
    for p, w in zip(student.parameters(), want):
        close("gradient", p.grad, w.double(), 4 * 2.0 ** -8)
