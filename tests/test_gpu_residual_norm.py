"""Residual norm, forward and backward, against the float64 oracle."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle.ref as R
import swish_activation_backward_amd as swg
from gpu_util import Guarded, device, note
from parity import to64
from residual_norm_models import bwd_models, fwd_models
from row_models import check

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
TYPES = [(BF16, BF16, BF16), (BF16, FP32, FP32), (BF16, FP32, BF16), (FP16, FP16, FP32),
         (FP16, FP32, FP16), (FP32, FP32, FP32)]
# one element, one lane, one wave, rows around the powers of two that a workgroup's vectors end
# at, odd widths, and rows longer than a workgroup's registers
SHAPES = [(1, 1), (3, 2), (5, 7), (7, 8), (4, 64), (33, 65), (1, 512), (130, 513), (9, 1023),
          (70, 1024), (6, 2047), (5, 2049), (1, 4096), (11, 4097), (3, 8192), (3, 8200),
          (2, 16384), (2, 16387), (1, 40001)]
GATES = ["none", "channel", "row", "full"]
PARTS = [(True, True), (False, True), (True, False), (False, False)]
EPS = 1e-6


def make(M, N, dt, rdt, wdt, gate="channel", seed=0, pad=0, shift=0):
    g = torch.Generator().manual_seed(1000 * seed + M + 7 * N)
    dev = device()

    def rows(t, s=1.0, cols=N):
        buf = torch.full((M * (cols + pad) + shift + 8,), float("nan"), dtype=t, device=dev)
        v = buf[shift:shift + M * (cols + pad)].view(M, cols + pad)[:, :cols]
        v.copy_((torch.randn(M, cols, generator=g) * s).to(t))
        return v

    d = {"y": rows(dt), "residual": rows(rdt), "dout": rows(rdt, 0.5), "dnorm": rows(dt, 0.5)}
    for n in ("w_post", "w_pre"):
        d[n] = (1 + 0.3 * torch.randn(N, generator=g)).to(wdt).to(dev)
    d["gate"] = {"none": lambda: None, "row": lambda: rows(dt, 1.0, 1), "full": lambda: rows(dt),
                 "channel": lambda: torch.randn(N, generator=g).to(wdt).to(dev)}[gate]()
    return d


def f64(t):
    return None if t is None else to64(t)


def check_fwd(d, r, scale, post=True, pre=True, residual="residual", eps=EPS):
    res = d[residual] if residual else None
    eps = float(np.float32(eps))
    ro, rn, rs, rp = R.residual_norm_ref(to64(d["y"]), f64(res), f64(d["w_post"]), f64(d["w_pre"]),
                                         f64(d["gate"]), scale, eps, post, pre)
    models = fwd_models(d["y"], res, d["w_post"], d["w_pre"], d["gate"], scale, rs, rp, ro)
    # what is not asked for is not there
    assert len(r) == 4
    for name, got, ref, e in zip(("out", "norm", "rstd_post", "rstd_pre"), r, (ro, rn, rs, rp),
                                 models):
        assert (got is None) == (ref is None), name
        if got is not None:
            check(name, got, ref, e)


def check_bwd(d, out, rstd_post, rstd_pre, scale, got, dout="dout", dnorm="dnorm", init=None):
    """``got``: dict of outputs; ``init``: contents that dw_post, dw_pre and dgate were added to."""
    a = (d[dout] if dout else None, d[dnorm] if dnorm else None, d["y"], out, d["w_post"],
         d["w_pre"], d["gate"], rstd_post, rstd_pre)
    ref = R.residual_norm_bwd_ref(*(f64(t) for t in a), scale)
    models = bwd_models(*a, scale)
    for name, r, e in zip(("dy", "dresidual", "dw_post", "dw_pre", "dgate"), ref, models):
        if got.get(name) is None:
            continue
        if init and name in init:
            r, e = r + to64(init[name]), e + 2.0 ** -24 * np.abs(to64(init[name]))
        check(name, got[name], r, e)


def grads(d, post, pre, M, N, dt, rdt, wdt, new):
    got = {"dy": new((M, N), dt), "dresidual": new((M, N), rdt)}
    if post:
        got["dw_post"] = new((N,), wdt)
    if pre:
        got["dw_pre"] = new((N,), wdt)
    if d["gate"] is not None:
        got["dgate"] = new(tuple(d["gate"].shape), d["gate"].dtype)
    return got


def run_both(d, M, N, dt, rdt, wdt, scale, post, pre):
    """Forward and backward between guard bands; returns nothing, checks everything."""
    dev = d["y"].device
    bands = []

    def new(shape, t):
        b = Guarded(shape, t, dev)
        bands.append(b)
        return b.t

    r = swg.residual_norm_fwd(
        d["y"], d["residual"], d["w_post"], d["w_pre"], d["gate"], scale, post, pre,
        out=new((M, N), rdt), norm=new((M, N), dt) if pre else None, stats=True,
        rstd_post=new((M,), FP32) if post else None, rstd_pre=new((M,), FP32) if pre else None,
        eps=EPS)
    got = grads(d, post, pre, M, N, dt, rdt, wdt, new)
    swg.residual_norm_bwd(d["dout"], d["dnorm"] if pre else None, d["y"], r.out, d["w_post"],
                          d["w_pre"], d["gate"], r.rstd_post, r.rstd_pre, scale=scale, **got)
    torch.cuda.synchronize()
    check_fwd(d, r, scale, post, pre)
    check_bwd(d, r.out, r.rstd_post, r.rstd_pre, scale, got, dnorm="dnorm" if pre else None)
    for b in bands:
        b.check()


@pytest.mark.parametrize("dt,rdt,wdt", TYPES)
@pytest.mark.parametrize("M,N", SHAPES)
def test_shapes_and_types(M, N, dt, rdt, wdt):
    gate = GATES[(M + N) % 4]
    note(f"residual norm M={M} N={N} {dt} {rdt} {wdt} {gate}")
    run_both(make(M, N, dt, rdt, wdt, gate), M, N, dt, rdt, wdt, 0.5, True, True)


@pytest.mark.parametrize("post,pre", PARTS)
@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("M,N", [(3, 5), (19, 200), (5, 1537), (3, 5000), (2, 17001)])
def test_parts_and_gates(M, N, gate, post, pre):
    note(f"residual norm M={M} N={N} gate={gate} post={post} pre={pre}")
    run_both(make(M, N, BF16, FP32, FP32, gate, seed=1), M, N, BF16, FP32, FP32, -1.25, post, pre)


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("pad,shift", [(8, 0), (1, 0), (3, 1), (43, 5)])
@pytest.mark.parametrize("N", [6, 96, 1001, 6000])
def test_strides_and_alignment(N, pad, shift, gate):
    M = 13
    note(f"residual norm N={N} pad={pad} shift={shift} gate={gate}")
    run_both(make(M, N, FP16, FP16, FP16, gate, seed=2, pad=pad, shift=shift), M, N, FP16, FP16,
             FP16, 1.0, True, True)


@pytest.mark.parametrize("post,pre", PARTS)
@pytest.mark.parametrize("N", [7, 24, 333, 1500, 3001, 9001, 20001])
def test_in_place(N, post, pre):
    """The new stream over the old one and its gradient over the incoming one: the same bits."""
    M = 37
    d = make(M, N, BF16, BF16, BF16, "channel", seed=3)
    a = swg.residual_norm_fwd(d["y"], d["residual"], d["w_post"], d["w_pre"], d["gate"], 0.5, post,
                              pre, stats=True, eps=EPS)
    stream = d["residual"].clone()
    b = swg.residual_norm_fwd(d["y"], stream, d["w_post"], d["w_pre"], d["gate"], 0.5, post, pre,
                              out=stream, stats=True, eps=EPS)
    assert b.out is stream
    both = []
    for src, dst in ((d["dout"], torch.empty(M, N, dtype=BF16, device=stream.device)),
                     ((t := d["dout"].clone()), t)):
        got = grads(d, post, pre, M, N, BF16, BF16, BF16,
                    lambda s, t: torch.empty(s, dtype=t, device=stream.device))
        got["dresidual"] = dst
        swg.residual_norm_bwd(src, d["dnorm"] if pre else None, d["y"], a.out, d["w_post"],
                              d["w_pre"], d["gate"], a.rstd_post, a.rstd_pre, scale=0.5, **got)
        both.append(got)
    torch.cuda.synchronize()
    for x, y in list(zip(a, b)) + [(both[0][k], both[1][k]) for k in both[0]]:
        assert (x is None and y is None) or torch.equal(x, y)


@pytest.mark.parametrize("N", [5, 257, 2048, 20000])
def test_optional_operands(N):
    """No weights, no residual, one incoming gradient at a time, single gradients wanted."""
    M, dev = 11, device()
    d = make(M, N, BF16, FP32, FP32, "full", seed=4)
    d["w_post"] = d["w_pre"] = None
    out = torch.empty(M, N, dtype=FP32, device=dev)
    r = swg.residual_norm_fwd(d["y"], None, gate=d["gate"], scale=2.0, out=out, stats=True, eps=EPS)
    check_fwd(d, r, 2.0, residual=None)
    for dout, dnorm in (("dout", None), (None, "dnorm"), (None, None)):
        for want in ("dy", "dresidual", "dw_post", "dw_pre", "dgate"):
            shape = (N,) if want.startswith("dw") else (M, N)
            t = FP32 if want in ("dw_post", "dw_pre", "dresidual") else BF16
            got = {"dy": None, "dresidual": None}
            got[want] = torch.full(shape, float("nan"), dtype=t, device=dev)
            swg.residual_norm_bwd(d[dout] if dout else None, d[dnorm] if dnorm else None, d["y"],
                                  r.out, None, None, d["gate"], r.rstd_post, r.rstd_pre, scale=2.0,
                                  **got)
            torch.cuda.synchronize()
            check_bwd(d, r.out, r.rstd_post, r.rstd_pre, 2.0, got, dout, dnorm)


@pytest.mark.parametrize("M", [0, 1, 300, 3000])
@pytest.mark.parametrize("N", [3, 40, 1030])
def test_accumulate(M, N):
    d = make(M, N, FP16, FP16, FP32, "channel", seed=5)
    dev = d["y"].device
    r = swg.residual_norm_fwd(d["y"], d["residual"], d["w_post"], d["w_pre"], d["gate"],
                              stats=True, eps=EPS)
    init = {n: torch.randn(N, device=dev) for n in ("dw_post", "dw_pre", "dgate")}
    for accumulate in (False, True):
        got = {n: t.clone() for n, t in init.items()}
        swg.residual_norm_bwd(d["dout"], d["dnorm"], d["y"], r.out, d["w_post"], d["w_pre"],
                              d["gate"], r.rstd_post, r.rstd_pre, None, None, accumulate=accumulate,
                              **got)
        torch.cuda.synchronize()
        if M == 0:   # the empty sums
            for n, t in got.items():
                assert torch.equal(t, init[n] if accumulate else torch.zeros_like(t))
        else:
            check_bwd(d, r.out, r.rstd_post, r.rstd_pre, 1.0, got,
                      init=init if accumulate else None)


def test_repeats_bit_for_bit():
    M, N = 5000, 768
    d = make(M, N, BF16, FP32, FP32, "channel", seed=6)
    first = None
    for _ in range(3):
        r = swg.residual_norm_fwd(d["y"], d["residual"], d["w_post"], d["w_pre"], d["gate"],
                                  stats=True)
        got = grads(d, True, True, M, N, BF16, FP32, FP32,
                    lambda s, t: torch.empty(s, dtype=t, device=r.out.device))
        swg.residual_norm_bwd(d["dout"], d["dnorm"], d["y"], r.out, d["w_post"], d["w_pre"],
                              d["gate"], r.rstd_post, r.rstd_pre, **got)
        torch.cuda.synchronize()
        now = [*r, *got.values()]
        first = first or now
        assert all(torch.equal(a, b) for a, b in zip(first, now))


@pytest.mark.parametrize("N", [4, 100, 3000])
def test_special_rows(N):
    """A row of zeros, one with a NaN and one with an infinity; the others keep their values."""
    M = 6
    d = make(M, N, FP32, FP32, FP32, "none", seed=7)
    want = swg.residual_norm_fwd(d["y"], d["residual"], d["w_post"], d["w_pre"], stats=True,
                                 eps=EPS)
    y, res = d["y"].clone(), d["residual"].clone()
    y[1] = 0
    res[1] = 0
    y[2, N // 2] = float("nan")
    res[4, 0] = float("inf")
    r = swg.residual_norm_fwd(y, res, d["w_post"], d["w_pre"], stats=True, eps=EPS)
    torch.cuda.synchronize()
    keep = [0, 3, 5]
    for a, b in zip(r, want):
        assert torch.equal(a[keep], b[keep])
    assert not r.out[1].any() and not r.norm[1].any()
    assert r.out[2].isnan().all() and r.norm[2].isnan().all()
    assert r.out[4, 0] == float("inf") and r.norm[4, 0].isnan()
    assert not r.norm[4, 1:].any()   # 1 / inf of finite values


def test_more_rows_than_workgroups():
    M, N = (1 << 20) + 3, 5
    g = torch.Generator(device="cuda").manual_seed(8)
    y = torch.randn(M, N, device="cuda", generator=g)
    r = swg.residual_norm_fwd(y, None, pre=False, eps=EPS)
    torch.cuda.synchronize()
    want = y.double() * (y.double().square().mean(1, keepdim=True) + EPS).rsqrt()
    # a root of a mean of 5 squares and two products: 16 roundings at most
    assert ((r.out.double() - want).abs() <= 16 * 2.0 ** -24 * want.abs()).all()
