"""Token log probabilities and distillation at the sizes where the library changes its way: rows
of many workgroups, rows held in registers, several tiles of a row, segments, and selections
whose bound leaves too many entries."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import oracle.ref as R
import swish_activation_backward_amd as swg
from gpu_util import Guarded, device, note
from parity import to64
from row_models import check, logit_errors
from test_gpu_vocab import (BF16, DTYPES, FP16, FP32, check_distill, check_logprobs,
                            check_logprobs_bwd, logits, targets_for, teacher)

pytestmark = pytest.mark.gpu


def spread(rows, n=9):
    """A few rows of many, the first and the last among them."""
    return sorted({int(i) for i in np.linspace(0, rows - 1, n)})


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("V", [3, 517, 2048, 2049, 8192, 8201, 16384, 20011, 32768, 40003, 65536,
                               70001, 131072, 131081])
def test_distill_in_one_call(V, dt):
    """256 rows and more; every row against the two calls, some against the oracle."""
    rows, k, T = 258, 12, 2.0
    note(f"distill one call V={V} {dt}")
    z = logits(rows, V, dt, seed=40)
    z[5] = math.nan
    z[6] = -math.inf
    z[7, : max(1, V // 2)] = -math.inf
    u, ids = teacher(rows, V, k)
    c = torch.rand(rows, device=z.device) + 0.5
    c[5] = 0.0
    ids[8] = -1
    dev = z.device
    loss, lse = Guarded((rows,), FP32, dev), Guarded((rows,), FP32, dev)
    dz = Guarded((rows, V), dt, dev)
    swg.distill_fwd_bwd(z, u, ids, c, dz.t, temperature=T, loss=loss.t, lse=lse.t)
    torch.cuda.synchronize()
    for o in (loss, lse, dz):
        o.check()
    rest = [r for r in [*spread(rows), 7, 8] if r not in (5, 6)]
    check_distill(z, u, ids, T, loss=loss.t, lse_out=lse.t, lse_in=lse.t, c=c, dz=dz.t, rows=rest)
    assert not bool(dz.t[5].any()) and bool(torch.isnan(loss.t[5]))
    assert not bool(dz.t[8].any()) and loss.t[8] == 0
    assert lse.t[6] == -math.inf
    # the other path agrees to within both roundings
    l2, s2 = swg.distill_fwd(z, u, ids, temperature=T)
    d2 = swg.distill_bwd(z, u, ids, lse.t, c, temperature=T)
    ok = [r for r in range(rows) if r not in (5, 6)]
    # |a| <= 16 here: a few hundred roundings of that size
    assert (s2[ok] - lse.t[ok]).abs().max() <= 2e-5
    assert torch.allclose(l2[ok], loss.t[ok], rtol=1e-5, atol=4 * 2e-5 * T * T)
    step = torch.finfo(dt).eps
    assert torch.allclose(d2[ok].float(), dz.t[ok].float(), rtol=step + 1e-5,
                          atol=1e-5 if dt == FP32 else float(torch.finfo(dt).tiny) + 1e-5)
    again = swg.distill_fwd_bwd(z, u, ids, c, temperature=T)
    for a, b in zip(again, (loss.t, lse.t, dz.t)):
        assert torch.equal(torch.nan_to_num(a), torch.nan_to_num(b))
    # in place
    swg.distill_fwd_bwd(z, u, ids, c, z, temperature=T)
    assert torch.equal(torch.nan_to_num(z), torch.nan_to_num(dz.t))


@pytest.mark.parametrize("pad,shift", [(1, 0), (5, 3), (64, 8)])
@pytest.mark.parametrize("V", [517, 9000, 70001])
@pytest.mark.parametrize("dt", [BF16, FP32])
def test_distill_in_one_call_strided(V, dt, pad, shift):
    rows, k = 300, 20
    note(f"distill one call strided V={V} {dt} pad={pad} shift={shift}")
    z = logits(rows, V, dt, seed=41, pad=pad, shift=shift)
    u, ids = teacher(rows, V, k, BF16)
    c = torch.rand(rows, device=z.device) + 0.5
    buf = torch.full((rows, V + 3), 7.0, dtype=dt, device=z.device)
    loss, lse, dz = swg.distill_fwd_bwd(z, u, ids, c, buf[:, :V], temperature=1.5)
    check_distill(z, u, ids, 1.5, loss=loss, lse_out=lse, lse_in=lse, c=c, dz=dz,
                  rows=spread(rows))
    assert bool((buf[:, V:] == 7).all())


@pytest.mark.parametrize("k", [1, 300, 1024])
@pytest.mark.parametrize("V", [60, 3000, 33000])
def test_distill_in_one_call_entries(V, k):
    """More entries than threads, and ids that repeat."""
    rows = 256
    note(f"distill one call entries V={V} k={k}")
    z = logits(rows, V, BF16, seed=42)
    u, ids = teacher(rows, V, k)
    c = torch.rand(rows, device=z.device) + 0.5
    loss, lse, dz = swg.distill_fwd_bwd(z, u, ids, c)
    check_distill(z, u, ids, 1.0, loss=loss, lse_out=lse, lse_in=lse, c=c, dz=dz,
                  rows=spread(rows))


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("V,top", [(500, 64), (4097, 20), (32768, 128), (32769, 5), (65537, 64),
                                   (140001, 33)])
def test_logprobs_of_many_rows(V, top, dt):
    """Rows that are not split: one workgroup a row, at 140001 in two tiles or more."""
    rows = 513
    note(f"logprobs many rows V={V} top={top} {dt}")
    z, t = logits(rows, V, dt, seed=43), targets_for(rows, V)
    z[7] = -math.inf
    z[9, 3:] = -math.inf
    r = swg.token_logprobs(z, t, top=top, temperature=0.8)
    sel = sorted({*spread(rows), 7, 9})
    check_logprobs(z[sel], t[sel], swg.TokenLogprobs(*(v[sel] for v in r)), 0.8, top)
    # the whole selection against torch's stable sort of a part of the rows
    part = slice(100, 140)
    ids = torch.sort(z[part].float(), dim=1, descending=True, stable=True).indices[:, :top]
    assert torch.equal(r.top_id[part], ids)


@pytest.mark.parametrize("rows", [13, 520])
@pytest.mark.parametrize("V", [3000, 20000, 140000])
@pytest.mark.parametrize("dt", [BF16, FP32])
def test_selection_where_bounds_fail(V, dt, rows):
    """Rising and falling rows (every entry of the best groups is a candidate), clusters, equal
    rows, an entry far above the rest, few usable entries, with 13 kinds of rows repeated."""
    top = 128
    g = torch.Generator().manual_seed(V)
    i = torch.arange(V, device=device(), dtype=torch.float32)
    n = torch.randn(V, generator=g).to(device())
    kinds = [i, -i, i / V - 0.5, (i // 32) * 1e-3, torch.zeros_like(i), torch.full_like(i, -1e4),
             torch.where(i == V // 3, 3e4, n), torch.where(i % 64 < 32, n + 50, n),
             torch.where(i < 200, n + 50, n), torch.where(i >= V - 130, n.abs() + 9, n),
             torch.where(i % 977 == 0, n, -math.inf), torch.where(i < 40, n, -math.inf),
             torch.where(i % 2 == 0, n, float(torch.finfo(dt).min))]
    z = torch.stack([kinds[r % 13] for r in range(rows)]).to(dt)
    note(f"selection V={V} {dt} rows={rows}")
    r = swg.token_logprobs(z, None, top=top)
    check_logprobs(z[:13], None, swg.TokenLogprobs(None, *(v[:13] for v in r[1:])), 1.0, top)
    for a in r[1:]:
        for c in range(13, rows, 13):
            m = min(13, rows - c)
            assert torch.equal(a[c:c + m], a[:m])


@pytest.mark.parametrize("V", [300, 5000, 140000])
@pytest.mark.parametrize("rows", [4, 514])
def test_nan_ranks_with_masked_entries(V, rows):
    """Fewer ordinary entries than asked for: NaN and -inf follow together by rising id."""
    top = 24
    z = torch.full((rows, V), -math.inf, dtype=BF16, device=device())
    z[:, V // 2] = 2.0
    z[:, V - 1] = 3.0
    z[:, 3] = math.nan
    z[1] = math.nan
    z[2, ::2] = math.nan
    note(f"nan order V={V} rows={rows}")
    ids = swg.token_logprobs(z, None, top=top).top_id[:4].cpu().numpy()
    want = R.top_ref(np.where(np.isnan(to64(z[:4])), -np.inf, to64(z[:4])), top)
    assert np.array_equal(ids, want)


@pytest.mark.parametrize("rows", [3, 300])
@pytest.mark.parametrize("V", [700, 9000, 140000])
def test_logits_near_the_types_range(V, rows):
    """Values whose quotient by T / log 2 leaves fp32, and whose differences stay in it."""
    z = logits(rows, V, FP32, seed=44)
    z[0] = torch.finfo(FP32).min
    z[1] = 3.1e38 + z[1] * 0
    z[2] = z[2] * 1e37
    note(f"range V={V} rows={rows}")
    sel = [0, 1, 2]
    r = swg.token_logprobs(z)
    z64 = to64(z[sel])
    lp, lse = R.log_softmax_ref(z64, 1.0)
    d = logit_errors(z[sel], 1.0, lp, lse)
    check("lse", r.lse[sel], lse, d.max(1))
    # one entry of row 2 takes everything, rows 0 and 1 are uniform
    ent = r.entropy[sel].cpu().numpy()
    assert np.allclose(ent, [math.log(V), math.log(V), 0.0], rtol=1e-5, atol=1e-6)
    u, ids = teacher(rows, V, 4, pads=False)
    c = torch.ones(rows, device=z.device)
    _, lse2, dz = swg.distill_fwd_bwd(z, u, ids, c)
    check("lse", lse2[sel], lse, d.max(1))
    hit = torch.zeros(rows, V, dtype=torch.bool, device=z.device)
    hit.scatter_(1, ids, True)
    # away from the teacher's entries the gradient of the uniform rows is 1 / V
    flat = dz[:2][~hit[:2]]
    assert torch.allclose(flat, torch.full_like(flat, 1.0 / V), rtol=1e-4)


@pytest.mark.parametrize("dt", [BF16, FP16])
@pytest.mark.parametrize("rows,V", [(1, 9000), (3, 140001), (300, 20011), (40, 70001)])
def test_gradients_of_segments(rows, V, dt):
    note(f"gradient segments R={rows} V={V} {dt}")
    z, t = logits(rows, V, dt, seed=45, pad=3, shift=1), targets_for(rows, V)
    r = swg.token_logprobs(z, t, temperature=1.3)
    g, h = torch.randn(2, rows, device=z.device)
    dz = swg.token_logprobs_bwd(z, t, r.lse, r.entropy, g, h, temperature=1.3)
    sel = spread(rows)
    pick = lambda a: a[sel]
    check_logprobs_bwd(z[sel], pick(t), pick(r.lse), pick(r.entropy), pick(g), pick(h), dz[sel],
                       1.3)
    u, ids = teacher(rows, V, 40)
    ids[0, :6] = torch.tensor([0, V - 1, V - 2, 1, 1, V - 1])   # a row's single elements, twice
    c = torch.rand(rows, device=z.device) + 0.5
    loss, lse = swg.distill_fwd(z, u, ids)
    dz = swg.distill_bwd(z, u, ids, lse, c)
    check_distill(z, u, ids, 1.0, loss=loss, lse_out=lse, lse_in=lse, c=c, dz=dz, rows=sel)


def test_more_rows_than_workgroups():
    """A launch holds 2^20 workgroups; the rows repeat with an odd period, so a row that a
    wrapped workgroup took for another would show.  Rows of 20 bf16 start at every other 8 bytes,
    and the order of a row's sums goes by that: two periods are compared with."""
    period, V, k = 1009, 20, 3
    rows = (1 << 20) + 5000
    note(f"rows {rows}")
    z1, t1 = logits(period, V, BF16, seed=46), targets_for(period, V)
    u1, ids1 = teacher(period, V, k)
    c1 = torch.rand(period, device=z1.device) + 0.5
    z1, t1, u1, ids1, c1 = (torch.cat((a, a)) for a in (z1, t1, u1, ids1, c1))
    i = torch.arange(rows, device=z1.device) % (2 * period)
    z, t, u, ids, c = (a[i].contiguous() for a in (z1, t1, u1, ids1, c1))
    r1, r = (swg.token_logprobs(a, b, top=k) for a, b in ((z1, t1), (z, t)))
    check_logprobs(z1, t1, r1, 1.0, k)
    for a, b in zip(r, r1):
        assert torch.equal(a, b[i])
    g1, h1 = torch.randn(2, 2 * period, device=z.device)
    d1 = swg.token_logprobs_bwd(z1, t1, r1.lse, r1.entropy, g1, h1)
    d = swg.token_logprobs_bwd(z, t, r.lse, r.entropy, g1[i], h1[i])
    assert torch.equal(d, d1[i])
    one, many = (swg.distill_fwd_bwd(*a) for a in ((z1, u1, ids1, c1), (z, u, ids, c)))
    check_distill(z1, u1, ids1, 1.0, loss=one[0], lse_out=one[1], lse_in=one[1], c=c1, dz=one[2])
    for a, b in zip(many, one):
        assert torch.equal(a, b[i])
    d1 = swg.distill_bwd(z1, u1, ids1, one[1], c1)
    d = swg.distill_bwd(z, u, ids, many[1], c)
    assert torch.equal(d, d1[i])
