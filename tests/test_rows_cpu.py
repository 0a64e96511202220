"""Layer norm, token log probabilities and distillation without a GPU: the C entry points'
refusals (no call here reaches a launch), the binding's checks, and the float64 oracle pinned
to torch's float64 gradients and to differences."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

import oracle.ref as R
import swish_activation_backward_amd as swg

OK, NULLPTR, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3, 4
BF16, FP16, FP32 = 0, 1, 2


def addr(i, off=0):
    """Fake device addresses 16 MiB apart: the checks must refuse before touching them."""
    return ctypes.c_void_p((i + 1) << 24 | off)


@pytest.fixture(scope="module")
def lib():
    return swg.load_library()


def norm_fwd(lib, **kw):
    a = dict(x=addr(0), ldx=64, w=addr(1), b=addr(2), y=addr(3), ldy=64, mean=addr(4),
             rstd=addr(5), M=8, N=64, eps=1e-5, dtype=BF16, wdtype=BF16)
    a.update(kw)
    return lib.layer_norm_fwd(*a.values(), None)


def norm_bwd(lib, **kw):
    a = dict(dy=addr(0), lddy=64, x=addr(1), ldx=64, w=addr(2), mean=addr(3), rstd=addr(4),
             dx=addr(5), lddx=64, dw=addr(6), db=addr(7), accumulate=0, M=8, N=64, dtype=BF16,
             wdtype=FP32, ws=addr(8), wsb=1 << 20)
    a.update(kw)
    return lib.layer_norm_bwd(*a.values(), None)


def logprobs(lib, **kw):
    a = dict(z=addr(0), ld=100, targets=addr(1), logprob=addr(2), entropy=addr(3), lse=addr(4),
             top_logprob=addr(5), top_id=addr(6), top=5, R=3, V=100, t=1.0, ignore=-100,
             dtype=BF16, ws=addr(7), wsb=1 << 24)
    a.update(kw)
    return lib.token_logprobs(*a.values(), None)


def logprobs_bwd(lib, **kw):
    a = dict(z=addr(0), ld=100, targets=addr(1), lse=addr(2), entropy=addr(3), g=addr(4),
             h=addr(5), dz=addr(6), ldd=100, R=3, V=100, t=1.0, ignore=-100, dtype=BF16)
    a.update(kw)
    return lib.token_logprobs_bwd(*a.values(), None)


def distill_fwd(lib, **kw):
    a = dict(z=addr(0), ld=100, u=addr(1), ids=addr(2), k=4, loss=addr(3), lse=addr(4), R=3,
             V=100, t=1.0, dtype=BF16, udtype=FP32, ws=addr(5), wsb=1 << 24)
    a.update(kw)
    return lib.distill_fwd(*a.values(), None)


def distill_bwd(lib, **kw):
    a = dict(z=addr(0), ld=100, u=addr(1), ids=addr(2), k=4, lse=addr(3), dloss=addr(4),
             dz=addr(5), ldd=100, R=3, V=100, t=1.0, dtype=BF16, udtype=FP32)
    a.update(kw)
    return lib.distill_bwd(*a.values(), None)


def distill_both(lib, **kw):
    a = dict(z=addr(0), ld=100, u=addr(1), ids=addr(2), k=4, dloss=addr(3), loss=addr(4),
             lse=addr(5), dz=addr(6), ldd=100, R=3, V=100, t=1.0, dtype=BF16, udtype=FP32,
             ws=addr(7), wsb=1 << 24)
    a.update(kw)
    return lib.distill_fwd_bwd(*a.values(), None)


REFUSALS = [
    (norm_fwd, INVALID, [dict(dtype=7), dict(wdtype=-1), dict(M=-1), dict(N=-1), dict(N=0),
                         dict(ldx=63), dict(ldy=10), dict(ldx=-64), dict(eps=-1e-5),
                         dict(eps=float("nan")), dict(eps=float("inf")), dict(x=addr(0, 1)),
                         dict(y=addr(3, 1)), dict(w=addr(1, 1)), dict(b=addr(2, 1)),
                         dict(mean=addr(4, 2)), dict(rstd=addr(5, 2)), dict(y=addr(0)),
                         dict(y=addr(0, 128)), dict(y=addr(1)), dict(mean=addr(0)),
                         dict(rstd=addr(4)), dict(M=1 << 31), dict(N=1 << 31, ldx=1 << 31),
                         dict(ldx=1 << 62, M=1 << 20)]),
    (norm_fwd, NULLPTR, [dict(x=None), dict(y=None)]),
    (norm_fwd, UNSUPPORTED, [dict(wdtype=FP16), dict(dtype=FP32, wdtype=BF16)]),
    (norm_fwd, OK, [dict(M=0), dict(M=0, N=0, ldx=0, ldy=0)]),
    (norm_bwd, INVALID, [dict(dtype=3), dict(M=-1), dict(N=0), dict(lddy=63), dict(ldx=63),
                         dict(lddx=63), dict(dy=addr(0, 1)), dict(dw=addr(6, 2)),
                         dict(mean=addr(3, 1)), dict(ws=addr(8, 8)), dict(dx=addr(0)),
                         dict(dx=addr(1)), dict(dw=addr(7)), dict(dw=addr(2)),
                         dict(db=addr(5)), dict(ws=addr(0)), dict(ws=addr(6))]),
    (norm_bwd, NULLPTR, [dict(dy=None), dict(x=None), dict(mean=None), dict(rstd=None),
                         dict(ws=None)]),
    (norm_bwd, UNSUPPORTED, [dict(wdtype=FP16)]),
    (norm_bwd, WORKSPACE, [dict(wsb=0), dict(wsb=64)]),
    (norm_bwd, OK, [dict(M=0, accumulate=1), dict(M=0, dw=None, db=None),
                    dict(dx=None, dw=None, db=None)]),
    (logprobs, INVALID, [dict(dtype=9), dict(R=-1), dict(V=-1), dict(V=0), dict(ld=99),
                         dict(top=-1), dict(top=101), dict(t=0.0), dict(t=-1.0),
                         dict(t=float("inf")), dict(t=float("nan")), dict(t=1e-45),
                         dict(z=addr(0, 1)), dict(targets=addr(1, 4)), dict(top_id=addr(6, 4)),
                         dict(lse=addr(4, 2)), dict(lse=addr(3)), dict(logprob=addr(0)),
                         dict(top_id=addr(1)), dict(R=1 << 31)]),
    (logprobs, NULLPTR, [dict(z=None), dict(targets=None), dict(logprob=None),
                         dict(top_id=None), dict(top_logprob=None)]),
    (logprobs, UNSUPPORTED, [dict(top=129, V=1000, ld=1000)]),
    (logprobs, OK, [dict(R=0)]),
    (logprobs_bwd, INVALID, [dict(dtype=9), dict(V=0), dict(ld=99), dict(ldd=99), dict(t=0.0),
                             dict(dz=addr(6, 1)), dict(dz=addr(0), ldd=101),
                             dict(dz=addr(0, 2)), dict(dz=addr(2)), dict(g=addr(4, 1)),
                             dict(dz=addr(5))]),
    (logprobs_bwd, NULLPTR, [dict(z=None), dict(lse=None), dict(dz=None), dict(targets=None),
                             dict(g=None), dict(entropy=None), dict(h=None)]),
    (logprobs_bwd, OK, [dict(R=0)]),
    (distill_fwd, INVALID, [dict(dtype=9), dict(udtype=9), dict(V=0), dict(ld=99), dict(k=0),
                            dict(t=0.0), dict(u=addr(1, 2)), dict(ids=addr(2, 4)),
                            dict(loss=addr(4)), dict(lse=addr(1)), dict(loss=addr(3, 1))]),
    (distill_fwd, NULLPTR, [dict(z=None), dict(u=None), dict(ids=None), dict(loss=None)]),
    (distill_fwd, UNSUPPORTED, [dict(k=1025)]),
    (distill_fwd, OK, [dict(R=0)]),
    (distill_bwd, INVALID, [dict(k=0), dict(ldd=99), dict(dz=addr(0), ldd=101),
                            dict(dz=addr(1)), dict(dz=addr(4)), dict(dloss=addr(4, 2)),
                            dict(dz=addr(5, 1))]),
    (distill_bwd, NULLPTR, [dict(z=None), dict(lse=None), dict(dloss=None), dict(dz=None)]),
    (distill_bwd, UNSUPPORTED, [dict(k=1025)]),
    (distill_bwd, OK, [dict(R=0)]),
    (distill_both, INVALID, [dict(k=0), dict(ldd=99), dict(dz=addr(0), ldd=101),
                             dict(loss=addr(0)), dict(loss=addr(0), dz=addr(0)),
                             dict(lse=addr(3)), dict(dz=addr(0, 2))]),
    (distill_both, NULLPTR, [dict(loss=None), dict(lse=None), dict(dloss=None), dict(dz=None)]),
    (distill_both, UNSUPPORTED, [dict(k=1025)]),
    (distill_both, OK, [dict(R=0)]),
]


@pytest.mark.parametrize("call,status,changes", REFUSALS,
                         ids=[f"{c.__name__}-{swg.STATUS[s]}" for c, s, _ in REFUSALS])
def test_refusals(lib, call, status, changes):
    for kw in changes:
        assert call(lib, **kw) == status, kw


def test_workspace_queries():
    bf = torch.bfloat16
    assert swg.layer_norm_bwd_workspace_size(0, 64, bf) == 0
    assert swg.layer_norm_bwd_workspace_size(-1, 64, bf) == 0
    assert swg.layer_norm_bwd_workspace_size(1, 64, bf) >= 2 * 64 * 4
    assert swg.token_logprobs_workspace_size(0, 64, 1, bf) == 0
    assert swg.token_logprobs_workspace_size(1, 64, 65, bf) == 0
    assert swg.distill_workspace_size(1, 64, 0, bf) == 0
    # sizes stay bounded: partials are a fraction of what they summarise
    for M, N in ((220000, 512), (16384, 4096), (1 << 20, 64), (64, 1 << 20)):
        assert swg.layer_norm_bwd_workspace_size(M, N, bf) <= max(M * N, 16 * N)
    for rows in (1, 3, 100, 5000):
        for V in (1, 100, 50021, 131072, 1 << 20):
            assert swg.token_logprobs_workspace_size(rows, V, min(V, 128), bf) <= 64 << 20


# ------------------------------------------------------------------ the binding's checks
def test_binding_refuses_before_the_library():
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    f = torch.zeros(4)
    ids = torch.zeros(4, 2, dtype=torch.int64)
    with pytest.raises(ValueError, match="GPU only"):
        swg.layer_norm_fwd(x, None, None)
    with pytest.raises(ValueError, match="GPU only"):
        swg.token_logprobs(x)
    with pytest.raises(ValueError, match="GPU only"):
        swg.distill_fwd(x, f[:, None].repeat(1, 2), ids)
    with pytest.raises(ValueError, match="two dimensions"):
        swg.layer_norm_fwd(x[0], None, None)
    with pytest.raises(ValueError, match="unsupported dtype"):
        swg.layer_norm_fwd(x.double(), None, None)
    with pytest.raises(ValueError, match="strides"):
        swg.layer_norm_fwd(x.t(), None, None)
    with pytest.raises(ValueError, match="strides"):
        swg.token_logprobs(x[:1].expand(4, 8))
    with pytest.raises(ValueError, match="shape"):
        swg.layer_norm_fwd(x, torch.ones(7, dtype=torch.bfloat16), None)
    with pytest.raises(ValueError, match="dtype"):
        swg.layer_norm_fwd(x, torch.ones(8), torch.ones(8, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="dtype"):
        swg.token_logprobs(x, torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError, match="shape"):
        swg.token_logprobs(x, torch.zeros(3, dtype=torch.int64))
    with pytest.raises(TypeError):
        swg.token_logprobs_bwd(x, None, None, None, None, None)
    with pytest.raises(ValueError, match="dtype"):
        swg.distill_fwd(x, f[:, None].repeat(1, 2), ids.int())
    with pytest.raises(ValueError, match="shape"):
        swg.distill_bwd(x, torch.zeros(4, 3), ids, f, f)


# ------------------------------------------------------------------ the oracle's pins
def test_layer_norm_oracle_matches_autograd():
    g = torch.Generator().manual_seed(3)
    x, dy = (torch.randn(5, 9, generator=g, dtype=torch.float64) for _ in range(2))
    w, b = (torch.randn(9, generator=g, dtype=torch.float64) for _ in range(2))
    for t in (x, w, b):
        t.requires_grad_()
    y = torch.nn.functional.layer_norm(x, (9,), w, b, 1e-5)
    y.backward(dy)
    ry, mean, rstd = R.layer_norm_ref(x.detach(), w.detach(), b.detach(), 1e-5)
    assert np.allclose(ry, y.detach().numpy(), rtol=1e-12, atol=1e-13)
    dx, dw, db = R.layer_norm_bwd_ref(dy, x.detach(), w.detach(), mean, rstd)
    for got, t in ((dx, x), (dw, w), (db, b)):
        assert np.allclose(got, t.grad.numpy(), rtol=1e-11, atol=1e-12)


def test_logprob_oracle_matches_autograd():
    g = torch.Generator().manual_seed(4)
    z = torch.randn(4, 11, generator=g, dtype=torch.float64) * 3
    z[1, ::3] = -torch.inf
    z.requires_grad_()
    t, T = torch.tensor([0, 4, 10, 3]), 0.7
    gl, h = torch.randn(2, 4, generator=g, dtype=torch.float64)
    lp = torch.log_softmax(z / T, 1)
    ent = torch.special.entr(lp.exp()).sum(1)
    taken = lp[torch.arange(4), t]
    # the entropy's gradient is formed from finite entries only
    keep = torch.isfinite(lp)
    p = lp.exp()
    ent2 = -(p[keep] * lp[keep]).new_zeros(4).index_add(
        0, keep.nonzero()[:, 0], p[keep] * lp[keep])
    (gl * taken + h * ent2).sum().backward()
    rlp, lse = R.log_softmax_ref(z.detach(), T)
    assert np.allclose(rlp, lp.detach().numpy(), rtol=1e-12, atol=1e-12)
    rent = R.entropy_ref(rlp)
    assert np.allclose(rent, ent.detach().numpy(), rtol=1e-12)
    d = R.token_logprobs_bwd_ref(z.detach(), T, t.numpy(), np.ones(4, bool), lse, rent, gl, h)
    assert np.allclose(d, z.grad.nan_to_num().numpy(), rtol=1e-10, atol=1e-12)


def test_distill_oracle_matches_autograd_and_differences():
    g = torch.Generator().manual_seed(5)
    z = (torch.randn(4, 13, generator=g, dtype=torch.float64) * 2).requires_grad_()
    u = torch.randn(4, 3, generator=g, dtype=torch.float64)
    ids = torch.tensor([[0, 5, 12], [1, 1, 2], [3, -1, 4], [13, -1, -7]])
    c, T = torch.rand(4, generator=g, dtype=torch.float64), 2.0
    keep = (ids >= 0) & (ids < 13)
    q = torch.softmax((u / T).masked_fill(~keep, -torch.inf)[:3], 1)
    lp = torch.log_softmax(z / T, 1)[:3].gather(1, ids[:3].clamp(0, 12))
    want = T * T * (torch.special.xlogy(q, q) - q * lp).sum(1)
    (c[:3] * want).sum().backward()
    loss, lse = R.distill_ref(z.detach(), T, u, ids.numpy())
    assert np.allclose(loss[:3], want.detach().numpy(), rtol=1e-12) and loss[3] == 0
    d = R.distill_bwd_ref(z.detach(), T, u, ids.numpy(), lse, c)
    assert np.allclose(d, z.grad.numpy(), rtol=1e-11, atol=1e-13)
    assert not d[3].any()
    eps = 1e-6
    for v in range(13):
        e = torch.zeros(13, dtype=torch.float64)
        e[v] = eps
        up, _ = R.distill_ref(z.detach() + e, T, u, ids.numpy())
        dn, _ = R.distill_ref(z.detach() - e, T, u, ids.numpy())
        assert np.allclose(c.numpy() * (up - dn) / (2 * eps), d[:, v], atol=1e-8)


def test_oracle_on_empty_rows_and_ties():
    z = np.array([[-np.inf] * 4, [1.0, 2.0, 2.0, -0.0], [0.0, -0.0, np.nan, -1.0]])
    lp, lse = R.log_softmax_ref(z, 1.0)
    assert np.isneginf(lse[0]) and np.isneginf(lp[0]).all() and R.entropy_ref(lp)[0] == 0
    assert R.top_ref(z, 4).tolist() == [[0, 1, 2, 3], [1, 2, 0, 3], [0, 1, 3, 2]]
