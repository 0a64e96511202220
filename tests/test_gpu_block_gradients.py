"""The autograd wrappers' gradients against the calls beneath them, bit by bit, and of one output of
the residual norm at a time, against float64."""
from __future__ import annotations

import pytest
import torch

import swish_activation_backward_amd as swg
from gpu_util import device
from swish_activation_backward_amd.autograd import Block, linear, residual_norm

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("act,beta", [("none", 1.0), ("relu", 1.0), ("swish", 1.7), ("gelu", 1.0),
                                      ("gelu_tanh", 1.0)])
@pytest.mark.parametrize("dt", [BF16, FP16, FP32])
def test_linear_is_its_calls(dt, act, beta, layout):
    g = torch.Generator().manual_seed(1)
    dev = device()
    rnd = lambda *s: torch.randn(*s, generator=g).to(dt).to(dev)  # noqa: E731
    x, b, res, dy = rnd(33, 40), rnd(24), rnd(33, 24), rnd(33, 24)
    w = rnd(40, 24) if layout == "kn" else rnd(24, 40).t()
    leaves = [t.detach().requires_grad_() for t in (x, w, b, res)]
    y = linear(*leaves, act, beta)
    got = torch.autograd.grad(y, leaves, dy)
    z, dx, db = torch.empty_like(dy), torch.empty_like(x), torch.empty_like(b)
    dw = torch.empty_like(w)                # of w's strides
    want = swg.linear_fwd(x, w, b, res, act, beta, z=z)
    swg.linear_bwd(dy, x, w, None if act == "none" else z, dx, dw, db, act, beta)
    torch.cuda.synchronize()
    for a, r in zip((y.detach(), *got), (want, dx, dw, db, dy)):
        assert torch.equal(a, r)


@pytest.mark.parametrize("used", ["out", "norm"])
@pytest.mark.parametrize("gate", ["none", "channel", "row", "full"])
def test_gradients_of_one_output(gate, used):
    g = torch.Generator().manual_seed(2)
    dev = device()
    rnd = lambda *s: torch.randn(*s, generator=g).to(dev)  # noqa: E731
    y, res, wp, wq, seed = rnd(9, 72), rnd(9, 72), 1 + rnd(72) / 5, 1 + rnd(72) / 5, rnd(9, 72)
    gv = {"none": lambda: None, "channel": lambda: rnd(72), "row": lambda: rnd(9, 1),
          "full": lambda: rnd(9, 72)}[gate]()
    leaves = [None if t is None else t.detach().requires_grad_() for t in (y, res, wp, wq, gv)]
    out, norm = residual_norm(*leaves, 0.5)
    want_wq = used == "norm"
    wanted = [t for i, t in enumerate(leaves) if t is not None and (i != 3 or want_wq)]
    got = torch.autograd.grad(out if used == "out" else norm, wanted, seed)
    d = [None if t is None else t.detach().double().requires_grad_() for t in leaves]
    yd, rd, wpd, wqd, gd = d
    u = yd * (yd.square().mean(-1, keepdim=True) + 1e-5).rsqrt() * wpd
    od = rd + 0.5 * (u if gd is None else u * gd)
    nd = od * (od.square().mean(-1, keepdim=True) + 1e-5).rsqrt() * wqd
    ref = torch.autograd.grad(od if used == "out" else nd,
                              [t for i, t in enumerate(d) if t is not None and (i != 3 or want_wq)],
                              seed.double())
    for i, (a, r) in enumerate(zip(got, ref)):
        # sums over 72 columns or 9 rows: under 200 roundings
        assert (a.double() - r).norm() <= 200 * 2.0 ** -24 * r.norm(), i
        assert r.norm() > 0.1


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
def test_block_is_its_calls(dtype):
    """Every gradient of a block, of a stream and a norm that both go on, from the calls in turn."""
    torch.manual_seed(4)
    dev = device()
    b = Block(64, 128, scale=0.5, device=dev, dtype=dtype)
    with torch.no_grad():
        for t in (b.w_post, b.w_pre, b.gate):
            t.add_(0.2 * torch.randn_like(t))
    s = torch.randn(10, 64, device=dev).requires_grad_()
    n = torch.randn(10, 64, device=dev).to(dtype).requires_grad_()
    out, norm = b(s, n)
    dout, dnorm = torch.randn_like(out), torch.randn(10, 64, device=dev).to(dtype)
    params = dict(b.named_parameters())
    got = torch.autograd.grad((out, norm), (s, n, *params.values()), (dout, dnorm))
    got = dict(zip(("s", "n", *params), got))
    with torch.no_grad():
        p = b.swiglu
        g, fc, h, dh, dg, dfc = (torch.empty(10, 128, dtype=dtype, device=dev) for _ in range(6))
        swg.swiglu_fwd(n, p.w_g, p.w_fc, p.b_g, p.b_fc, g, fc, h)
        y = swg.linear_fwd(h, b.out.w, b.out.b)
        r = swg.residual_norm_fwd(y, s, b.w_post, b.w_pre, b.gate, 0.5, stats=True)
        zeros = lambda t: torch.zeros_like(t)  # noqa: E731
        dy, want = torch.empty_like(y), {"s": torch.empty_like(s), "n": torch.empty_like(n)}
        want.update({k: zeros(t) for k, t in params.items()})
        swg.residual_norm_bwd(dout, dnorm, y, r.out, b.w_post, b.w_pre, b.gate, r.rstd_post,
                              r.rstd_pre, dy, want["s"], want["w_post"], want["w_pre"],
                              want["gate"], 0.5)
        swg.linear_bwd(dy, h, b.out.w, None, dh, want["out.w"], want["out.b"])
        swg.swiglu_bwd_b(dh, g, fc, dg, dfc, want["swiglu.b_g"], want["swiglu.b_fc"])
        swg.swiglu_bwd_wx(n, dg, dfc, p.w_g, p.w_fc, want["swiglu.w_g"], want["swiglu.w_fc"],
                          want["n"])
    torch.cuda.synchronize()
    for k in want:
        assert torch.equal(got[k], want[k]), k
