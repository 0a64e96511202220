"""Token log probabilities and distillation, forward and backward, against the float64
oracle."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import oracle.ref as R
import swish_activation_backward_amd as swg
from gpu_util import Guarded, device, note
from parity import to64
from row_models import (check, distill_bwd_model, distill_model, entropy_model, logit_errors,
                        logprobs_bwd_model, teacher_errors)

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
DTYPES = [BF16, FP16, FP32]
IGNORE = -100
# one entry, vector and wave borders, workgroup tiles, odd widths, long rows
WIDTHS = [1, 2, 7, 8, 15, 63, 64, 65, 500, 1000, 1023, 2048, 4096, 4097, 8191, 20000, 32000, 50021,
          131072, 151553, 300001]


def logits(rows, V, dt, seed=0, pad=0, shift=0, scale=2.0):
    g = torch.Generator().manual_seed(17 * seed + rows + 31 * V)
    buf = torch.full((rows * (V + pad) + shift + 8,), float("nan"), dtype=dt, device=device())
    z = buf[shift:shift + rows * (V + pad)].view(rows, V + pad)[:, :V]
    z.copy_((torch.randn(rows, V, generator=g) * scale).to(dt))
    return z


def targets_for(rows, V, seed=0):
    g = torch.Generator().manual_seed(seed + rows + V)
    t = torch.randint(0, V, (rows,), generator=g)
    if rows > 2:
        t[1] = IGNORE
    return t.to(device())


def check_logprobs(z, t, r, T, top, ignore=IGNORE):
    T = float(np.float32(T))
    z64 = to64(z)
    V = z64.shape[1]
    lp, lse = R.log_softmax_ref(z64, T)
    d = logit_errors(z, T, lp, lse)
    check("lse", r.lse, lse, d.max(1))
    check("entropy", r.entropy, R.entropy_ref(lp), entropy_model(lp, d))
    if t is not None:
        tt = t.cpu().numpy()
        at = np.clip(tt, 0, V - 1)
        rows = np.arange(len(tt))
        ref = np.where(tt == ignore, 0.0, lp[rows, at])
        ref[(tt != ignore) & ((tt < 0) | (tt >= V))] = np.nan
        check("logprob", r.logprob, ref, d[rows, at])
    if top:
        ids = R.top_ref(z64, top)
        assert r.top_id.dtype == torch.int64
        assert np.array_equal(r.top_id.cpu().numpy(), ids), "top_id"
        check("top_logprob", r.top_logprob, np.take_along_axis(lp, ids, 1),
              np.take_along_axis(d, ids, 1))
    return lp, lse, d


def check_logprobs_bwd(z, t, lse, ent, g, h, dz, T, ignore=IGNORE):
    T = float(np.float32(T))
    rows, V = z.shape
    tt = np.full(rows, ignore) if t is None else t.cpu().numpy()
    live = tt != ignore
    zero = np.zeros(rows)
    g64 = zero if g is None else to64(g)
    h64 = zero if h is None else to64(h)
    e64 = zero if ent is None else to64(ent)
    ref = R.token_logprobs_bwd_ref(to64(z), T, tt, live, to64(lse), e64, g64, h64)
    with np.errstate(invalid="ignore"):
        lp = np.where(np.isneginf(to64(z)), -np.inf, to64(z) / T - to64(lse)[:, None])
    d = logit_errors(z, T, lp, to64(lse))
    check("dlogits", dz, ref, logprobs_bwd_model(T, lp, d, np.where(live, g64, 0), h64, e64))


def teacher(rows, V, k, dt=FP32, seed=0, pads=True):
    """Entries in falling order at random (possibly repeated) ids, some rows padded."""
    g = torch.Generator().manual_seed(seed + rows + 3 * V + 5 * k)
    u = (8 + 2 * torch.randn(rows, k, generator=g)).sort(1, descending=True).values.to(dt)
    ids = torch.randint(0, V, (rows, k), generator=g)
    if pads and k > 2:
        ids[::3, k - 1] = -1
        ids[1::3, k - 2:] = V
    return u.to(device()), ids.to(device())


def check_distill(z, u, ids, T, loss=None, lse_out=None, lse_in=None, c=None, dz=None,
                  rows=None):
    T = float(np.float32(T))
    sel = slice(None) if rows is None else rows
    V = z.shape[1]
    z, u, ids = z[sel], u[sel], ids[sel]
    idn = ids.cpu().numpy()
    lp, lse = R.log_softmax_ref(to64(z), T)
    lq, q = R.teacher_ref(to64(u), idn, V, T)
    dq = teacher_errors(u, T, lq)
    at = np.clip(idn, 0, V - 1)
    if loss is not None:
        d = logit_errors(z, T, lp, lse)
        ref, _ = R.distill_ref(to64(z), T, to64(u), idn)
        check("loss", loss[sel], ref,
              distill_model(T, lq, q, np.take_along_axis(lp, at, 1),
                            np.take_along_axis(d, at, 1), dq))
        if lse_out is not None:
            check("lse", lse_out[sel], lse, d.max(1))
    if dz is not None:
        ls = to64(lse_in[sel]) if lse_in is not None else lse
        ref = R.distill_bwd_ref(to64(z), T, to64(u), idn, ls, to64(c[sel]))
        with np.errstate(invalid="ignore"):
            lp = np.where(np.isneginf(to64(z)), -np.inf, to64(z) / T - ls[:, None])
        d = logit_errors(z, T, lp, ls)
        check("dlogits", dz[sel], ref,
              distill_bwd_model(to64(z), T, idn, np.exp(lp), d, q, dq, to64(c[sel])))


# ------------------------------------------------------------------ token log probabilities
@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("V", WIDTHS)
def test_logprobs(V, dt):
    for rows, top, T in ((1, min(20, V), 1.0), (5, min(64, V), 0.7), (3, 0, 2.5)):
        note(f"token_logprobs R={rows} V={V} top={top} T={T} {dt}")
        z, t = logits(rows, V, dt), targets_for(rows, V)
        dev = z.device
        outs = [Guarded((rows,), FP32, dev) for _ in range(3)]
        tl = Guarded((rows, max(top, 1)), FP32, dev)
        out = swg.TokenLogprobs(outs[0].t, outs[1].t, outs[2].t, tl.t if top else None, None)
        r = swg.token_logprobs(z, t, top=top, temperature=T, out=out)
        torch.cuda.synchronize()
        lp, lse, d = check_logprobs(z, t, r, T, top)
        for o in outs + [tl]:
            o.check()
        note(f"token_logprobs_bwd R={rows} V={V} T={T} {dt}")
        g = torch.randn(rows, device=dev)
        h = torch.randn(rows, device=dev) * 0.1
        dz = Guarded((rows, V), dt, dev)
        swg.token_logprobs_bwd(z, t, r.lse, r.entropy, g, h, dz.t, temperature=T)
        torch.cuda.synchronize()
        check_logprobs_bwd(z, t, r.lse, r.entropy, g, h, dz.t, T)
        dz.check()


@pytest.mark.parametrize("top", [1, 2, 33, 100, 128])
@pytest.mark.parametrize("V", [128, 129, 1000, 9999, 70001, 131072])
def test_top_counts(V, top):
    rows = 3
    note(f"top counts V={V} top={top}")
    for dt in (BF16, FP32):
        z = logits(rows, V, dt, seed=1)
        r = swg.token_logprobs(z, None, top=top)
        assert r.logprob is None
        check_logprobs(z, None, r, 1.0, top)


@pytest.mark.parametrize("V", [64, 1000, 16384, 50021, 131072, 262145])
@pytest.mark.parametrize("dt", [BF16, FP32])
def test_top_where_order_goes_wrong(V, dt):
    """Rows of equal entries, sorted rows, rows whose largest entries sit at one place of every
    tile, both zeros, and values of both signs: equal entries come by rising id."""
    top = 64
    i = torch.arange(V, device=device())
    base = torch.full((V,), -3.0, device=device())
    rows = [torch.zeros(V, device=device()), i.float() / V * 8, -(i.float()) / V * 8]
    for period, at in ((4096, 16), (4096, 4095), (16, 0), (1024, 7), (8192, 8000), (64, 63)):
        rows.append(torch.where(i % period == at % period, 5.0, base))
    for lo in (0, max(0, V - 200), V // 2):
        rows.append(torch.where((i >= lo) & (i < lo + 150), 1.0 + (i % 3).float(), base))
    z0 = torch.zeros(V, device=device())
    z0[::2] = -0.0
    rows.append(z0)
    rows.append(torch.where(i % 97 == 5, 0.25, -torch.rand(V, device=device())))
    z = torch.stack(rows).to(dt)
    note(f"top order V={V} {dt}")
    r = swg.token_logprobs(z, None, top=top)
    check_logprobs(z, None, r, 1.0, top)


@pytest.mark.parametrize("V", [40, 1000, 33000, 140001])
@pytest.mark.parametrize("dt", DTYPES)
def test_masked_rows(V, dt):
    """-inf entries, rows that keep one entry or fewer alternatives than asked for, rows that
    keep none, and the type's lowest value as a mask."""
    rows, top = 7, 32
    z = logits(rows, V, dt, seed=2)
    i = torch.arange(V, device=z.device)
    z[0, i % 3 != 0] = -math.inf
    z[1] = -math.inf
    z[2] = -math.inf
    z[2, V // 2] = 1.5
    z[3, 10:] = -math.inf
    z[4, i % 2 == 0] = torch.finfo(dt).min
    z[5] = torch.finfo(dt).min
    z[6] = -math.inf
    t = torch.tensor([1, 3, V // 2, 9, 1, 0, IGNORE], device=z.device)
    note(f"masked rows V={V} {dt}")
    r = swg.token_logprobs(z, t, top=top)
    lp, lse, d = check_logprobs(z, t, r, 1.0, top)
    assert r.lse[1] == -math.inf and r.logprob[1] == -math.inf and r.entropy[1] == 0
    assert r.logprob[6] == 0 and bool((r.top_logprob[1] == -math.inf).all())
    g, h = torch.randn(2, rows, device=z.device)
    dz = swg.token_logprobs_bwd(z, t, r.lse, r.entropy, g, h)
    check_logprobs_bwd(z, t, r.lse, r.entropy, g, h, dz, 1.0)
    u, ids = teacher(rows, V, 4, pads=False)
    ids[:] = torch.tensor([0, 3, 6, 9], device=z.device)   # kept by rows 0 and 3
    ids[2] = V // 2
    c = torch.rand(rows, device=z.device) + 0.5
    for loss, lse2, dz in (
            (*swg.distill_fwd(z, u, ids), swg.distill_bwd(z, u, ids, r.lse, c)),
            swg.distill_fwd_bwd(z, u, ids, c)):
        check_distill(z, u, ids, 1.0, loss=loss, lse_out=lse2, lse_in=r.lse, c=c, dz=dz)
        assert loss[1] == math.inf


def test_nan_and_infinite_logits():
    """They make their own row's values NaN and no other's."""
    for V in (100, 5000, 140000):
        z = logits(4, V, BF16, seed=3)
        z[1, V // 2] = math.nan
        z[2, V - 1] = math.inf
        t = torch.tensor([0, 1, 2, 3], device=z.device)
        r = swg.token_logprobs(z, t, top=8)
        for row in (1, 2):
            assert all(bool(torch.isnan(v[row]).all())
                       for v in (r.logprob, r.entropy, r.lse, r.top_logprob))
        ok = [0, 3]
        check_logprobs(z[ok], t[ok], swg.TokenLogprobs(*(v[ok] for v in r)), 1.0, 8)
        for row in (1, 2):
            ids = r.top_id[row].tolist()
            assert len(set(ids)) == 8 and min(ids) >= 0 and max(ids) < V
        assert r.top_id[2, 0] == V - 1


def test_targets_outside_the_vocabulary():
    V = 3001
    z = logits(5, V, BF16, seed=4)
    t = torch.tensor([V, -1, IGNORE, 7, 1 << 40], device=z.device)
    r = swg.token_logprobs(z, t)
    check_logprobs(z, t, r, 1.0, 0)
    g = torch.ones(5, device=z.device)
    dz = swg.token_logprobs_bwd(z, t, r.lse, None, g, None)
    assert bool(torch.isnan(dz[[0, 1, 4]]).all()) and not bool(dz[2].any())
    check_logprobs_bwd(z[3:4], t[3:4], r.lse[3:4], None, g[3:4], None, dz[3:4], 1.0)
    r2 = swg.token_logprobs(z, t, ignore_index=7)
    assert r2.logprob[3] == 0 and bool(torch.isnan(r2.logprob[2]))


@pytest.mark.parametrize("pad,shift", [(0, 1), (1, 0), (8, 0), (43, 3), (5, 7)])
@pytest.mark.parametrize("V", [700, 32768, 50021])
@pytest.mark.parametrize("dt", DTYPES)
def test_row_strides_and_alignment(V, dt, pad, shift):
    rows = 4
    note(f"vocab strided V={V} pad={pad} shift={shift} {dt}")
    z, t = logits(rows, V, dt, seed=5, pad=pad, shift=shift), targets_for(rows, V)
    r = swg.token_logprobs(z, t, top=10)
    check_logprobs(z, t, r, 1.0, 10)
    g, h = torch.randn(2, rows, device=z.device)
    buf = torch.full((rows, V + pad), 7.0, dtype=dt, device=z.device)
    swg.token_logprobs_bwd(z, t, r.lse, r.entropy, g, h, buf[:, :V])
    check_logprobs_bwd(z, t, r.lse, r.entropy, g, h, buf[:, :V], 1.0)
    assert bool((buf[:, V:] == 7).all())
    u, ids = teacher(rows, V, 12)
    c = torch.rand(rows, device=z.device) + 0.5
    buf.fill_(7.0)
    loss, lse, dz = swg.distill_fwd_bwd(z, u, ids, c, buf[:, :V], temperature=2.0)
    check_distill(z, u, ids, 2.0, loss=loss, lse_out=lse, lse_in=lse, c=c, dz=dz)
    assert bool((buf[:, V:] == 7).all())
    # in place: every gradient may take the logits' own storage
    keep = z.clone()
    l2, s2, d2 = swg.distill_fwd_bwd(z, u, ids, c, z, temperature=2.0)
    assert d2 is z and torch.equal(z, dz) and torch.equal(l2, loss) and torch.equal(s2, lse)
    z.copy_(keep)
    swg.distill_bwd(z, u, ids, lse, c, z, temperature=2.0)
    check_distill(keep, u, ids, 2.0, lse_in=lse, c=c, dz=z)
    z.copy_(keep)
    swg.token_logprobs_bwd(z, t, r.lse, r.entropy, g, h, z)
    check_logprobs_bwd(keep, t, r.lse, r.entropy, g, h, z, 1.0)


@pytest.mark.parametrize("which", ["logprob", "entropy", "neither"])
def test_bwd_optional_operands(which):
    rows, V = 3, 999
    z, t = logits(rows, V, FP32, seed=6), targets_for(rows, V)
    r = swg.token_logprobs(z, t)
    g = torch.randn(rows, device=z.device) if which == "logprob" else None
    h = torch.randn(rows, device=z.device) if which == "entropy" else None
    tt, ent = (t if g is not None else None), (r.entropy if h is not None else None)
    dz = swg.token_logprobs_bwd(z, tt, r.lse, ent, g, h)
    check_logprobs_bwd(z, tt, r.lse, ent, g, h, dz, 1.0)


@pytest.mark.parametrize("rows,V", [(2000, 517), (1500, 4100), (700, 20011), (5000, 64)])
def test_many_rows(rows, V):
    note(f"vocab many rows R={rows} V={V}")
    z, t = logits(rows, V, BF16, seed=7), targets_for(rows, V)
    r = swg.token_logprobs(z, t, top=3)
    check_logprobs(z, t, r, 1.0, 3)
    again = swg.token_logprobs(z, t, top=3)
    assert all(torch.equal(a, b) for a, b in zip(r, again))
    g, h = torch.randn(2, rows, device=z.device)
    dz = swg.token_logprobs_bwd(z, t, r.lse, r.entropy, g, h)
    check_logprobs_bwd(z, t, r.lse, r.entropy, g, h, dz, 1.0)
    u, ids = teacher(rows, V, 9)
    c = torch.rand(rows, device=z.device)
    loss, lse, dz = swg.distill_fwd_bwd(z, u, ids, c)
    check_distill(z, u, ids, 1.0, loss=loss, lse_out=lse, lse_in=lse, c=c, dz=dz)


def test_offsets_past_32_bits():
    """Rows more than 2^31 elements apart."""
    V, ld = 3000, (1 << 31) // 2 + 8
    buf = torch.empty(2 * ld + V, dtype=BF16, device=device())
    z = torch.as_strided(buf, (3, V), (ld, 1))
    src = logits(3, V, BF16, seed=8)
    z.copy_(src)
    t = targets_for(3, V)
    r = swg.token_logprobs(z, t, top=5)
    check_logprobs(src, t, r, 1.0, 5)
    g, h = torch.randn(2, 3, device=z.device)
    u, ids = teacher(3, V, 6)
    c = torch.ones(3, device=z.device)
    loss, lse, dz = swg.distill_fwd_bwd(z, u, ids, c)
    check_distill(src, u, ids, 1.0, loss=loss, lse_out=lse, lse_in=lse, c=c, dz=dz)
    swg.token_logprobs_bwd(z, t, r.lse, r.entropy, g, h, z)
    check_logprobs_bwd(src, t, r.lse, r.entropy, g, h, z, 1.0)


# ------------------------------------------------------------------ distillation
@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("V", WIDTHS)
def test_distill(V, dt):
    for rows, k, T in ((1, 16, 1.0), (5, 64, 2.0), (4, 3, 4.0)):
        note(f"distill R={rows} V={V} k={k} T={T} {dt}")
        z = logits(rows, V, dt, seed=9)
        u, ids = teacher(rows, V, k)
        dev = z.device
        loss, lse = Guarded((rows,), FP32, dev), Guarded((rows,), FP32, dev)
        dz = Guarded((rows, V), dt, dev)
        c = torch.rand(rows, device=dev) + 0.1
        swg.distill_fwd(z, u, ids, temperature=T, loss=loss.t, lse=lse.t)
        swg.distill_bwd(z, u, ids, lse.t, c, dz.t, temperature=T)
        torch.cuda.synchronize()
        check_distill(z, u, ids, T, loss=loss.t, lse_out=lse.t, lse_in=lse.t, c=c, dz=dz.t)
        for o in (loss, lse, dz):
            o.check()
            o.t.fill_(7.0)
        swg.distill_fwd_bwd(z, u, ids, c, dz.t, temperature=T, loss=loss.t, lse=lse.t)
        torch.cuda.synchronize()
        check_distill(z, u, ids, T, loss=loss.t, lse_out=lse.t, lse_in=lse.t, c=c, dz=dz.t)
        for o in (loss, lse, dz):
            o.check()


@pytest.mark.parametrize("k", [1, 2, 63, 65, 257, 1000, 1024])
@pytest.mark.parametrize("udt", DTYPES)
@pytest.mark.parametrize("V", [50, 5000, 40000])
def test_distill_entries(V, udt, k):
    """Every entry count and teacher type; ids repeat (V = 50 holds each many times)."""
    rows = 4
    note(f"distill entries V={V} k={k} {udt}")
    z = logits(rows, V, BF16, seed=10)
    u, ids = teacher(rows, V, k, udt)
    c = torch.rand(rows, device=z.device) + 0.1
    loss, lse = swg.distill_fwd(z, u, ids, temperature=1.5)
    dz = swg.distill_bwd(z, u, ids, lse, c, temperature=1.5)
    check_distill(z, u, ids, 1.5, loss=loss, lse_out=lse, lse_in=lse, c=c, dz=dz)
    loss, lse, dz = swg.distill_fwd_bwd(z, u, ids, c, temperature=1.5)
    check_distill(z, u, ids, 1.5, loss=loss, lse_out=lse, lse_in=lse, c=c, dz=dz)


@pytest.mark.parametrize("V", [200, 9000, 140000])
def test_distill_padding_and_masked_rows(V):
    """Rows of padding only, teacher entries of -inf, one entry, weight 0 over a row of NaN."""
    rows, k = 6, 8
    z = logits(rows, V, BF16, seed=11)
    u, ids = teacher(rows, V, k, pads=False)
    ids[0] = -1
    ids[1] = torch.tensor([V, -5, 1 << 40, -(1 << 40), V + 1, -1, -100, V * 2], device=z.device)
    u[2] = -math.inf
    u[3, 1:] = -math.inf
    z[4] = math.nan
    c = torch.rand(rows, device=z.device) + 0.5
    c[4] = 0.0
    ok = [0, 1, 2, 3, 5]
    loss, lse = swg.distill_fwd(z, u, ids)
    dz = swg.distill_bwd(z, u, ids, lse, c)
    l2, s2, d2 = swg.distill_fwd_bwd(z, u, ids, c)
    for lo, ls, d in ((loss, lse, dz), (l2, s2, d2)):
        check_distill(z, u, ids, 1.0, loss=lo, lse_out=ls, lse_in=ls, c=c, dz=d, rows=ok)
        assert not bool(lo[:3].any()) and not bool(d[:3].any())
        assert not bool(d[4].any()) and bool(torch.isnan(lo[4]))


def test_distill_gradient_is_the_losses_derivative():
    """dlogits against central differences of the oracle's loss in float64."""
    rows, V, k, T = 3, 40, 6, 1.5
    z = logits(rows, V, FP32, seed=12)
    u, ids = teacher(rows, V, k)
    c = torch.rand(rows, device=z.device) + 0.5
    _, _, dz = swg.distill_fwd_bwd(z, u, ids, c, temperature=T)
    z64, u64, idn = to64(z), to64(u), ids.cpu().numpy()
    got, h = to64(dz), 1e-5
    for v in range(V):
        e = np.zeros(V)
        e[v] = h
        up, _ = R.distill_ref(z64 + e, T, u64, idn)
        dn, _ = R.distill_ref(z64 - e, T, u64, idn)
        # central difference: h^2 times a third derivative of order 1, and rounding / h
        assert np.abs(to64(c) * (up - dn) / (2 * h) - got[:, v]).max() <= 1e-6


def test_logprob_gradient_is_the_derivative():
    rows, V, T = 3, 40, 0.8
    z = logits(rows, V, FP32, seed=13)
    t = torch.tensor([0, 39, 7], device=z.device)
    r = swg.token_logprobs(z, t, temperature=T)
    g, h = torch.randn(2, rows, device=z.device)
    dz = to64(swg.token_logprobs_bwd(z, t, r.lse, r.entropy, g, h, temperature=T))
    z64, tt, eps = to64(z), t.cpu().numpy(), 1e-5

    def value(a):
        lp, _ = R.log_softmax_ref(a, float(np.float32(T)))
        return to64(g) * lp[np.arange(rows), tt] + to64(h) * R.entropy_ref(lp)

    for v in range(V):
        e = np.zeros(V)
        e[v] = eps
        diff = (value(z64 + e) - value(z64 - e)) / (2 * eps)
        assert np.abs(diff - dz[:, v]).max() <= 4e-6


def test_other_stream_and_graph():
    """On a stream of its own, and captured into a graph that replays with new inputs; the
    small row count takes the split path."""
    for rows, V in ((2, 70001), (300, 4100)):
        z, t = logits(rows, V, BF16, seed=14), targets_for(rows, V)
        u, ids = teacher(rows, V, 8)
        c = torch.rand(rows, device=z.device)
        r = swg.token_logprobs(z, t, top=7)
        dz1, dz2 = torch.empty_like(z), torch.empty_like(z)
        loss, lse, _ = swg.distill_fwd_bwd(z, u, ids, c, dz2)
        n1 = swg.token_logprobs_workspace_size(rows, V, 7, BF16)
        n2 = swg.distill_workspace_size(rows, V, 8, BF16)
        w1, w2 = (torch.empty(max(n, 16), dtype=torch.uint8, device=z.device) for n in (n1, n2))
        g, h = torch.randn(2, rows, device=z.device)

        def step(stream=None):
            swg.token_logprobs(z, t, top=7, out=r, workspace=w1, stream=stream)
            swg.token_logprobs_bwd(z, t, r.lse, r.entropy, g, h, dz1, stream=stream)
            swg.distill_fwd_bwd(z, u, ids, c, dz2, loss=loss, lse=lse, workspace=w2,
                                stream=stream)

        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        step(side)
        torch.cuda.current_stream().wait_stream(side)
        check_logprobs(z, t, r, 1.0, 7)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for i in range(4):
            z.copy_(logits(rows, V, BF16, seed=30 + i))
            graph.replay()
            torch.cuda.synchronize()
            got = [x.clone() for x in (*r, dz1, dz2, loss, lse)]
            step()
            torch.cuda.synchronize()
            for a, b in zip(got, (*r, dz1, dz2, loss, lse)):
                assert torch.equal(a, b)
