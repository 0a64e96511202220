"""Linear layer without a GPU: the C entry points' refusals (no call here reaches a launch), the
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
NAN, INF = float("nan"), float("inf")


def addr(i, off=0):
    """Fake device addresses 16 MiB apart: the checks must refuse before touching them."""
    return ctypes.c_void_p((i + 1) << 24 | off)


@pytest.fixture(scope="module")
def lib():
    return swg.load_library()


def fwd(lib, **kw):
    a = dict(x=addr(0), ldx=64, w=addr(1), ldw=128, nk=0, bias=addr(2), r=addr(3), ldr=128,
             y=addr(4), ldy=128, z=addr(5), ldz=128, M=8, K=64, N=128, act=3, beta=1.0, dtype=BF16,
             ws=addr(6), wsb=1 << 22)
    a.update(kw)
    return lib.linear_fwd(*a.values(), None)


def bwd(lib, **kw):
    a = dict(dy=addr(0), lddy=128, x=addr(1), ldx=64, w=addr(2), ldw=128, nk=0, z=addr(3), ldz=128,
             dx=addr(4), lddx=64, dw=addr(5), lddw=128, db=addr(6), accumulate=0, M=8, K=64, N=128,
             act=3, beta=1.0, dtype=BF16, ws=addr(7), wsb=1 << 22)
    a.update(kw)
    return lib.linear_bwd(*a.values(), None)


REFUSALS = [
    (fwd, INVALID, [dict(dtype=5), dict(act=5), dict(act=-1), dict(beta=NAN), dict(beta=INF),
                    dict(M=-1), dict(K=-1), dict(N=-1), dict(ldx=63), dict(ldw=127),
                    dict(nk=1, ldw=63), dict(ldr=127), dict(ldy=127), dict(ldz=127),
                    dict(x=addr(0, 1)), dict(w=addr(1, 1)), dict(bias=addr(2, 1)),
                    dict(r=addr(3, 1)), dict(y=addr(4, 1)), dict(z=addr(5, 1)), dict(y=addr(0)),
                    dict(y=addr(1)), dict(y=addr(2)), dict(y=addr(3, 2)),
                    dict(y=addr(3), ldy=136), dict(z=addr(3)), dict(z=addr(4)), dict(z=addr(0)),
                    dict(M=1 << 31), dict(ldx=1 << 62, M=1 << 20)]),
    (fwd, NULLPTR, [dict(x=None), dict(w=None), dict(y=None)]),
    (fwd, UNSUPPORTED, [dict(K=1 << 22, ldx=1 << 22), dict(N=1 << 22, ldw=1 << 22, ldy=1 << 22,
                                                           ldr=1 << 22, ldz=1 << 22)]),
    (fwd, OK, [dict(M=0), dict(N=0), dict(M=0, x=None, y=None)]),
    (bwd, INVALID, [dict(dtype=5), dict(act=7), dict(beta=NAN), dict(M=-1), dict(K=-1),
                    dict(N=-1), dict(lddy=127), dict(ldx=63), dict(ldw=127), dict(nk=1, ldw=63),
                    dict(ldz=127), dict(lddx=63), dict(lddw=127), dict(nk=1, lddw=63),
                    dict(dy=addr(0, 1)), dict(x=addr(1, 1)), dict(w=addr(2, 1)),
                    dict(z=addr(3, 1)), dict(dx=addr(4, 1)), dict(dw=addr(5, 1)),
                    dict(db=addr(6, 1)), dict(dx=addr(0)), dict(dx=addr(2)), dict(dw=addr(1)),
                    dict(dw=addr(4)), dict(db=addr(5)), dict(db=addr(3)), dict(dx=addr(3)),
                    dict(ws=addr(0)), dict(ws=addr(4)), dict(ws=addr(7, 8))]),
    (bwd, NULLPTR, [dict(dy=None), dict(x=None), dict(w=None), dict(z=None), dict(ws=None)]),
    (bwd, WORKSPACE, [dict(wsb=0), dict(wsb=64)]),
    (bwd, UNSUPPORTED, [dict(K=1 << 22, ldx=1 << 22, lddx=1 << 22)]),
    (bwd, OK, [dict(M=0, accumulate=1), dict(dx=None, dw=None, db=None), dict(M=0, dw=None, db=None),
               dict(N=0, dx=None), dict(K=0, db=None)]),
]


@pytest.mark.parametrize("call,status,changes", REFUSALS,
                         ids=[f"{c.__name__}-{swg.STATUS[s]}" for c, s, _ in REFUSALS])
def test_refusals(lib, call, status, changes):
    for kw in changes:
        assert call(lib, **kw) == status, kw


def test_workspace_queries():
    bf = torch.bfloat16
    for bad in ((0, 8, 8), (8, 8, 0), (-1, 8, 8), (8, 1 << 22, 8)):
        assert swg.linear_bwd_workspace_size(*bad, bf) == 0
        assert swg.linear_fwd_workspace_size(*bad, bf) == 0
    # room for the operands that have to be laid out again covers the case that none has to
    for M, K, N in ((1, 64, 64), (300, 1000, 1001), (5000, 256, 264), (65, 31, 33)):
        for nk in (False, True):
            assert (swg.linear_fwd_workspace_size(M, K, N, bf, nk, rows16=False)
                    >= swg.linear_fwd_workspace_size(M, K, N, bf, nk, rows16=True))
            assert (swg.linear_bwd_workspace_size(M, K, N, bf, "gelu", nk, rows16=False)
                    >= swg.linear_bwd_workspace_size(M, K, N, bf, "gelu", nk, rows16=True))


@pytest.fixture
def t():
    with FakeTensorMode():
        f = lambda *s, dt=torch.bfloat16: torch.empty(*s, dtype=dt, device="cuda:0")  # noqa: E731
        yield SimpleNamespace(f=f, x=f(4, 8), w=f(8, 16), y=f(4, 16))


def test_binding_refuses(t):
    f32 = torch.float32
    bad = [dict(x=t.f(8)), dict(x=t.f(4, 8, dt=torch.int32)), dict(x=t.f(8, 4).t()),
           dict(w=t.f(7, 16)), dict(w=t.f(8, 16, dt=f32)), dict(w=t.f(8, 32)[:, ::2]),
           dict(w=t.f(8)), dict(w=t.f(1, 16).expand(8, 16)), dict(bias=t.f(8)),
           dict(bias=t.f(32)[::2]), dict(bias=t.f(16, dt=f32)), dict(residual=t.f(4, 8)),
           dict(residual=t.f(1, 16).expand(4, 16)), dict(y=t.f(4, 16, dt=f32)), dict(z=t.f(4, 15)),
           dict(act="tanh"), dict(act=None), dict(x=torch.empty(4, 8, dtype=torch.bfloat16))]
    for kw in bad:
        a = dict(x=t.x, w=t.w)
        a.update(kw)
        with pytest.raises(ValueError):
            swg.linear_fwd(**a)
    for kw in (dict(x=None), dict(w=3.0)):
        a = dict(x=t.x, w=t.w)
        a.update(kw)
        with pytest.raises(TypeError):
            swg.linear_fwd(**a)


def test_binding_refuses_backward(t):
    bad = [dict(act="gelu"), dict(act="swish", z=t.f(4, 8)), dict(x=None), dict(w=None),
           dict(dw=t.f(16, 8).t()), dict(dw=t.f(16, 8)), dict(dx=t.f(4, 16)), dict(db=t.f(8)),
           dict(dy=t.f(3, 16)), dict(dy=t.f(16))]
    for kw in bad:
        a = dict(dy=t.y, x=t.x, w=t.w, z=None, dx=t.f(4, 8), dw=t.f(8, 16), db=t.f(16))
        a.update(kw)
        with pytest.raises(ValueError):
            swg.linear_bwd(**a)


def test_other_devices_stream_is_refused(t):
    s = SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=1)
    with pytest.raises(ValueError, match="stream of cuda:1"):
        swg.linear_fwd(t.x, t.w, stream=s)
    with pytest.raises(ValueError, match="stream of cuda:1"):
        swg.linear_bwd(t.y, t.x, t.w, None, None, t.f(8, 16), stream=s)


@pytest.mark.parametrize("act,beta", [("none", 1.0), ("relu", 1.0), ("swish", 1.0),
                                      ("swish", -1.7), ("gelu", 1.0), ("gelu_tanh", 1.0)])
def test_oracle_gradients(act, beta):
    g = torch.Generator().manual_seed(5)
    rnd = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    x, w, b, res, dy = rnd(5, 6), rnd(6, 7), rnd(7), rnd(5, 7), rnd(5, 7)
    fn = {"none": lambda z: z, "relu": torch.relu, "swish": lambda z: z * torch.sigmoid(beta * z),
          "gelu": torch.nn.functional.gelu,
          "gelu_tanh": lambda z: torch.nn.functional.gelu(z, approximate="tanh")}[act]

    def loss(x, w, b):
        return ((fn(x @ w + b) + res) * dy).sum()

    leaves = [v.requires_grad_() for v in (x, w, b)]
    want = torch.autograd.grad(loss(*leaves), leaves)
    n = lambda v: v.detach().numpy()  # noqa: E731
    y, z = R.linear_ref(n(x), n(w), n(b), n(res), act, beta)
    np.testing.assert_allclose(y, n(fn(x @ w + b) + res), rtol=1e-12, atol=1e-14)
    dx, dw, db, _ = R.linear_bwd_ref(n(dy), n(x), n(w), z, act, beta)
    for got, v in zip((dx, dw, db), want):
        np.testing.assert_allclose(got, v.numpy(), rtol=1e-11, atol=1e-12)
    with torch.no_grad():
        for v, got in ((x, dx), (w, dw), (b, db)):
            step, base = rnd(*v.shape), v.clone()
            v.copy_(base + 1e-5 * step)
            up = loss(x, w, b)
            v.copy_(base - 1e-5 * step)
            down = loss(x, w, b)
            v.copy_(base)
            # central differences: an error of the order of the step's square
            assert abs(float((up - down) / 2e-5) - float((step.numpy() * got).sum())) < 1e-7


def test_a_token_against_contiguous_columns_needs_no_workspace():
    bf, f32 = torch.bfloat16, torch.float32
    for dt in (bf, f32):
        assert swg.linear_fwd_workspace_size(1, 4096, 4096, dt, True) == 0
        assert swg.linear_fwd_workspace_size(16, 1001, 77, dt, True) == 0
    # one row of tiles that would leave most of the chip idle is split, and joined from there
    assert swg.linear_fwd_workspace_size(1, 16384, 64, bf, True) > 0
    assert swg.linear_fwd_workspace_size(17, 4096, 4096, bf, True) > 0


def test_row_limit(lib):
    most = (1 << 31) - 1024
    wide = dict(x=addr(0), w=None, y=None, z=None)
    assert fwd(lib, M=most, **wide) == UNSUPPORTED
    assert fwd(lib, M=most - 1, **wide) == NULLPTR
    assert bwd(lib, M=most, dy=None) == UNSUPPORTED
    assert bwd(lib, M=most - 1, dy=None) == NULLPTR
