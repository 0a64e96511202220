"""Residual norm without a GPU: the C entry points' refusals (no call here reaches a launch), the
binding's checks, and the float64 oracle against torch's float64 gradients and differences."""
from __future__ import annotations

import ctypes
from types import SimpleNamespace

import numpy as np
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import oracle.ref as R
import swish_activation_backward_amd as swg

OK, NULLPTR, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3, 4
BF16, FP16, FP32 = 0, 1, 2
NONE, CHANNEL, ROW, FULL = range(4)


def addr(i, off=0):
    """Fake device addresses 16 MiB apart: the checks must refuse before touching them."""
    return ctypes.c_void_p((i + 1) << 24 | off)


@pytest.fixture(scope="module")
def lib():
    return swg.load_library()


def fwd(lib, **kw):
    a = dict(y=addr(0), ldy=64, r=addr(1), ldr=64, wp=addr(2), wq=addr(3), gate=addr(4), ldg=64,
             kind=FULL, scale=1.0, out=addr(5), ldo=64, norm=addr(6), ldn=64, rs=addr(7),
             rp=addr(8), post=1, pre=1, M=8, N=64, eps=1e-5, dtype=BF16, rdtype=FP32, wdtype=BF16)
    a.update(kw)
    return lib.residual_norm_fwd(*a.values(), None)


def bwd(lib, **kw):
    a = dict(dout=addr(0), lddo=64, dnorm=addr(1), lddn=64, y=addr(2), ldy=64, out=addr(3), ldo=64,
             wp=addr(4), wq=addr(5), gate=addr(6), ldg=64, kind=FULL, scale=1.0, rs=addr(7),
             rp=addr(8), dy=addr(9), lddy=64, dr=addr(10), lddr=64, dwp=addr(11), dwq=addr(12),
             dgate=addr(13), lddg=64, accumulate=0, M=8, N=64, dtype=BF16, rdtype=FP32,
             wdtype=FP32, ws=addr(14), wsb=1 << 20)
    a.update(kw)
    return lib.residual_norm_bwd(*a.values(), None)


NAN, INF = float("nan"), float("inf")
REFUSALS = [
    (fwd, INVALID, [dict(dtype=7), dict(rdtype=-1), dict(wdtype=9), dict(kind=4), dict(kind=-1),
                    dict(M=-1), dict(N=-1), dict(N=0), dict(ldy=63), dict(ldr=63), dict(ldo=63),
                    dict(ldn=63), dict(ldg=63), dict(kind=ROW, ldg=0), dict(eps=-1e-5),
                    dict(eps=NAN), dict(eps=INF), dict(scale=NAN), dict(scale=-INF),
                    dict(y=addr(0, 1)), dict(r=addr(1, 2)), dict(out=addr(5, 2)),
                    dict(norm=addr(6, 1)), dict(wp=addr(2, 1)), dict(wq=addr(3, 1)),
                    dict(gate=addr(4, 1)), dict(wdtype=FP32, kind=CHANNEL, gate=addr(4, 2)),
                    dict(rs=addr(7, 2)), dict(rp=addr(8, 1)), dict(out=addr(0)),
                    dict(out=addr(1, 4)), dict(out=addr(1), ldo=65), dict(norm=addr(1)),
                    dict(norm=addr(5)), dict(norm=addr(0)), dict(out=addr(4)), dict(rs=addr(8)),
                    dict(rp=addr(2)), dict(M=1 << 31), dict(N=1 << 31, ldy=1 << 31),
                    dict(ldy=1 << 62, M=1 << 20)]),
    (fwd, NULLPTR, [dict(y=None), dict(out=None), dict(norm=None), dict(gate=None),
                    dict(kind=CHANNEL, gate=None)]),
    (fwd, UNSUPPORTED, [dict(wdtype=FP16), dict(rdtype=FP16), dict(dtype=FP32, wdtype=BF16),
                        dict(dtype=FP32, wdtype=FP32, rdtype=BF16)]),
    (fwd, OK, [dict(M=0), dict(M=0, N=0), dict(M=0, y=None, out=None)]),
    (bwd, INVALID, [dict(dtype=3), dict(rdtype=3), dict(wdtype=3), dict(kind=4), dict(M=-1),
                    dict(N=0), dict(lddo=63), dict(lddn=63), dict(ldy=63), dict(ldo=63),
                    dict(lddy=63), dict(lddr=63), dict(ldg=63), dict(lddg=63), dict(scale=NAN),
                    dict(rs=None), dict(rp=None), dict(rp=None, dwq=None),
                    dict(rp=None, dnorm=None), dict(kind=NONE), dict(dout=addr(0, 2)),
                    dict(dnorm=addr(1, 1)), dict(y=addr(2, 1)), dict(out=addr(3, 2)),
                    dict(wp=addr(4, 2)), dict(gate=addr(6, 1)), dict(dgate=addr(13, 1)),
                    dict(rs=addr(7, 2)), dict(dy=addr(9, 1)), dict(dr=addr(10, 2)),
                    dict(dwp=addr(11, 2)), dict(ws=addr(14, 8)), dict(dy=addr(2)),
                    dict(dy=addr(10)), dict(dr=addr(0, 4)), dict(dr=addr(0), lddr=65),
                    dict(dr=addr(3)), dict(dwp=addr(12)), dict(dwp=addr(4)), dict(dgate=addr(6)),
                    dict(ws=addr(0)), dict(ws=addr(11)), dict(M=1 << 31)]),
    (bwd, NULLPTR, [dict(y=None), dict(out=None), dict(gate=None), dict(ws=None)]),
    (bwd, UNSUPPORTED, [dict(wdtype=FP16), dict(rdtype=FP16)]),
    (bwd, WORKSPACE, [dict(wsb=0), dict(wsb=64)]),
    (bwd, OK, [dict(M=0, accumulate=1), dict(M=0, dwp=None, dwq=None),
               dict(dy=None, dr=None, dwp=None, dwq=None, dgate=None)]),
]


@pytest.mark.parametrize("call,status,changes", REFUSALS,
                         ids=[f"{c.__name__}-{swg.STATUS[s]}" for c, s, _ in REFUSALS])
def test_refusals(lib, call, status, changes):
    for kw in changes:
        assert call(lib, **kw) == status, kw


def test_workspace_queries():
    bf = torch.bfloat16
    assert swg.residual_norm_bwd_workspace_size(0, 64, bf) == 0
    assert swg.residual_norm_bwd_workspace_size(8, 0, bf) == 0
    assert swg.residual_norm_bwd_workspace_size(-1, 64, bf) == 0
    assert swg.residual_norm_bwd_workspace_size(1, 1, bf) > 0
    # bounded by a few hundred partial rows, whatever the batch
    assert swg.residual_norm_bwd_workspace_size(1 << 24, 512, bf) <= (1 << 27) + 512 * 8 * 2048


@pytest.fixture
def t():
    with FakeTensorMode():
        f = lambda *s, dt=torch.bfloat16: torch.empty(*s, dtype=dt, device="cuda:0")  # noqa: E731
        yield SimpleNamespace(
            f=f, y=f(4, 8), r=f(4, 8, dt=torch.float32), w=f(8, dt=torch.float32),
            s=f(4, dt=torch.float32))


def test_binding_refuses(t):
    f32 = torch.float32
    bad = [
        dict(y=t.f(8)), dict(y=t.f(4, 8, dt=torch.int32)), dict(residual=t.f(4, 9)),
        dict(residual=t.f(8, 4).t()), dict(w_post=t.f(7, dt=f32)), dict(w_pre=t.f(8)),
        dict(gate=t.f(4)), dict(gate=t.f(4, 2)), dict(gate=t.f(8)), dict(gate=t.f(4, 1, dt=f32)),
        dict(gate=t.f(4, 8, dt=f32)), dict(out=t.f(4, 8)), dict(norm=t.f(4, 8, dt=f32)),
        dict(stats=True, rstd_post=t.f(5, dt=f32)), dict(stats=True, rstd_pre=t.f(4)), dict(residual=torch.empty(4, 8)),
        dict(gate=torch.empty(4, 8, dtype=torch.bfloat16)),
    ]
    for kw in bad:
        a = dict(y=t.y, residual=t.r, w_post=t.w, w_pre=t.w, gate=None)
        a.update(kw)
        with pytest.raises(ValueError):
            swg.residual_norm_fwd(**a)
    for kw in (dict(y=None), dict(residual=1.0), dict(gate=0.5)):
        a = dict(y=t.y, residual=t.r, gate=None)
        a.update(kw)
        with pytest.raises(TypeError):
            swg.residual_norm_fwd(**a)


def test_binding_refuses_backward(t):
    f32 = torch.float32
    bad = [
        dict(dout=t.f(4, 8)), dict(dnorm=t.f(4, 8, dt=f32)), dict(dnorm=t.f(3, 8)),
        dict(out=None), dict(rstd_pre=None), dict(dy=t.f(4, 8, dt=f32)), dict(dresidual=t.f(4, 8)),
        dict(dw_post=t.f(8)), dict(dgate=t.f(8, dt=f32)), dict(gate=t.f(4, 1), dgate=t.f(4, 8)),
        dict(rstd_post=t.f(4)),
    ]
    for kw in bad:
        a = dict(dout=t.r, dnorm=t.y, y=t.y, out=t.r, w_post=t.w, w_pre=t.w, gate=None,
                 rstd_post=t.s, rstd_pre=t.s, dy=t.y, dresidual=t.r)
        a.update(kw)
        with pytest.raises(ValueError):
            swg.residual_norm_bwd(**a)


def test_other_devices_stream_is_refused(t):
    s = SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=1)
    with pytest.raises(ValueError, match="stream of cuda:1"):
        swg.residual_norm_fwd(t.y, t.r, stream=s)
    with pytest.raises(ValueError, match="stream of cuda:1"):
        swg.residual_norm_bwd(t.r, None, t.y, None, None, None, None, t.s, None, t.y, t.r, stream=s)


@pytest.mark.parametrize("post,pre", [(True, True), (False, True), (True, False), (False, False)])
@pytest.mark.parametrize("gate", ["none", "channel", "row", "full"])
def test_oracle_gradients(gate, post, pre):
    """Against torch's float64 gradients through the statistics, and against differences."""
    g = torch.Generator().manual_seed(3)
    M, N, scale, eps = 5, 7, -0.75, 1e-3
    rnd = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    y, res, dout, dnorm = rnd(M, N), rnd(M, N), rnd(M, N), rnd(M, N)
    wp, wq = 1 + 0.2 * rnd(N), 1 + 0.2 * rnd(N)
    gv = {"none": None, "channel": rnd(N), "row": rnd(M, 1), "full": rnd(M, N)}[gate]

    def loss(y, res, wp, wq, gv):
        u = y * (y.square().mean(1, keepdim=True) + eps).rsqrt() * wp if post else y
        out = res + scale * (u if gv is None else u * gv)
        total = (out * dout).sum()
        if pre:
            total = total + (out * (out.square().mean(1, keepdim=True) + eps).rsqrt() * wq
                             * dnorm).sum()
        return total

    leaves = [t.requires_grad_() for t in (y, res, wp, wq)]
    if gv is not None:
        leaves.append(gv.requires_grad_())
    want = torch.autograd.grad(loss(y, res, wp, wq, gv), leaves, allow_unused=True)
    n = lambda t: None if t is None else t.detach().numpy()  # noqa: E731
    out, _, rs, rp = R.residual_norm_ref(n(y), n(res), n(wp), n(wq), n(gv), scale, eps, post, pre)
    dy, dr, dwp, dwq, dg = R.residual_norm_bwd_ref(
        n(dout), n(dnorm) if pre else None, n(y), out, n(wp), n(wq), n(gv), rs, rp, scale)
    for got, w in zip((dy, dr, dwp, dwq, dg), want):
        if w is None or got is None:
            assert got is None or w is None
            continue
        np.testing.assert_allclose(got, w.numpy(), rtol=1e-11, atol=1e-12)
    # differences: central, step 1e-5, error of the order of its square
    with torch.no_grad():
        for t, got in ((y, dy), (res, dr)):
            v = rnd(M, N)
            base = t.clone()
            t.copy_(base + 1e-5 * v)
            up = loss(y, res, wp, wq, gv)
            t.copy_(base - 1e-5 * v)
            down = loss(y, res, wp, wq, gv)
            t.copy_(base)
            assert abs(float((up - down) / 2e-5) - float((v.numpy() * got).sum())) < 1e-7
