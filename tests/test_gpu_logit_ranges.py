"""Logits far from the ordinary range: large finite masks, rows of large values, tiny
temperatures, values whose difference leaves fp32, signaling NaN, and gradients
from an lse that is too coarse for them; the same of a teacher's values."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import oracle.ref as R
import swish_activation_backward_amd as swg
from gpu_util import device, note
from logit_range_models import check_forward, check_loss
from parity import to64
from row_models import U
from test_gpu_vocab import BF16, DTYPES, FP16, FP32, logits, teacher

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ rows of large equal values
@pytest.mark.parametrize("dt", [BF16, FP32])
@pytest.mark.parametrize("value", [1e5, 1e6, 1e7, 1e8, -1e5, -1e6, -1e7, -1e8])
def test_rows_of_large_equal_values(value, dt):
    """log p = -log V whatever the value and wherever the row starts: single elements at a row's
    ends and its chunks have one reference."""
    note(f"equal values {value} {dt}")
    for V in (1, 2, 7, 14, 23, 300, 4099, 9001):
        buf = torch.full((3 * V + 8,), value, dtype=dt, device=device())
        for shift in range(8):
            z = buf[shift:shift + 3 * V].view(3, V)
            t = torch.tensor([0, V // 2, V - 1], device=z.device)
            r = swg.token_logprobs(z, t, top=min(V, 5))
            check_forward(z, t, r, 1.0, min(V, 5))
            u, ids = teacher(3, V, 2, pads=False)
            loss, lse = swg.distill_fwd(z, u, ids)
            check_loss(z, u, ids, 1.0, loss, lse)
            c = torch.ones(3, device=z.device)
            loss, lse, dz = swg.distill_fwd_bwd(z, u, ids, c)
            check_loss(z, u, ids, 1.0, loss, lse, c, dz)


# ------------------------------------------------------------------ large finite masks
MASKS = [(-1e8, 1.0), (-1e9, 1.0), (-1e9, 0.1), (-1e10, 1.0), (-1e10, 2.0), (-1e12, 1.0),
         (-1e15, 2.0), (-1e20, 1.0), (-1e20, 0.1), (-1e25, 1.0), (-1e30, 2.0), (-1e30, 0.1)]
# one workgroup a row, segments, rows held in registers, two tiles
FORMS = [(3000, 7), (20000, 7), (20000, 518), (131072, 7), (131072, 518), (140001, 518)]


def masked_kinds(V, dt, mask, seed=0):
    """Seven rows: the first third masked, the last third, everything, everything but one entry,
    every second entry, every second chunk, and masked entries beside -inf."""
    z = logits(7, V, dt, seed=seed).clone()
    i = torch.arange(V, device=z.device)
    z[0, : V // 3] = mask
    z[1, V - V // 3:] = mask
    z[2] = mask
    z[3] = mask
    z[3, V // 2] = 1.5
    z[4, i % 2 == 0] = mask
    z[5, i // 8 % 2 == 0] = mask
    z[6] = -math.inf
    z[6, : V // 2] = mask
    return z


@pytest.mark.parametrize("dt", [BF16, FP32])
@pytest.mark.parametrize("V,rows", FORMS)
def test_large_finite_masks(V, rows, dt):
    top, k = 20, 6
    for mask, T in MASKS if V < 100000 else MASKS[2:4] + MASKS[7:11:3]:
        note(f"mask {mask} T={T} V={V} rows={rows} {dt}")
        kinds = masked_kinds(V, dt, mask)
        i = torch.arange(rows, device=kinds.device) % 7
        z = kinds[i].contiguous()
        t = torch.tensor([1, V - 2, 3, V // 2, 5, 9, 4], device=z.device)
        r = swg.token_logprobs(z, t[i], top=top, temperature=T)
        check_forward(kinds, t, swg.TokenLogprobs(*(v[:7] for v in r)), T, top)
        u, ids = teacher(7, V, k, pads=False)
        c = torch.rand(7, device=z.device) + 0.5
        loss, lse = swg.distill_fwd(z, u[i], ids[i], temperature=T)
        check_loss(kinds, u, ids, T, loss[:7], lse[:7])
        both = swg.distill_fwd_bwd(z, u[i], ids[i], c[i], temperature=T)
        check_loss(kinds, u, ids, T, both[0][:7], both[1][:7], c, both[2][:7])
        for a in (*r, loss, lse, *both):
            assert not bool(torch.isnan(a).any())


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("T", [1e-3, 1e-6, 1e-9, 1e-30])
@pytest.mark.parametrize("V,rows", [(3000, 5), (20000, 5), (20000, 518), (140001, 5)])
def test_tiny_temperatures(V, rows, dt, T):
    """Ordinary logits: almost all of a row's probability lies on its largest entries."""
    note(f"temperature {T} V={V} rows={rows} {dt}")
    z = logits(rows, V, dt, seed=50)
    t = z.float().argmax(1)
    r = swg.token_logprobs(z, t, top=9, temperature=T)
    check_forward(z[:5], t[:5], swg.TokenLogprobs(*(v[:5] for v in r)), T, 9)
    # a teacher of one entry (loss = -T^2 log p) and weights that keep T^2 and c T in range
    u = torch.zeros(rows, 1, device=z.device)
    c = torch.full((rows,), min(1.0 / T, 1e30), device=z.device)
    both = swg.distill_fwd_bwd(z, u, t[:, None].contiguous(), c, temperature=T)
    check_loss(z[:5], u[:5], t[:5, None], T, both[0][:5], both[1][:5], c[:5], both[2][:5])


# ------------------------------------------------------------------ selections
@pytest.mark.parametrize("dt", [BF16, FP32])
@pytest.mark.parametrize("V,rows", [(131072, 3), (131072, 515), (30000, 515), (20000, 3)])
def test_selection_over_a_range_beyond_fp32(V, rows, dt):
    """The largest entry less the type's lowest value leaves fp32; few groups hold any entry
    that is not masked."""
    top, n = 20, 26
    low = torch.finfo(dt).min
    z = torch.full((rows, V), -math.inf, dtype=dt, device=device())
    at = torch.arange(n, device=z.device) * (V // n) + 3 * torch.arange(n, device=z.device)
    z[:, at] = low
    z[:, at[5::10]] = 3e38
    z[1] = -math.inf          # other ids than the rows around it
    z[1, at + 1] = low
    z[1, at[2::9] + 1] = 2e38
    note(f"selection range V={V} rows={rows} {dt}")
    got = swg.token_logprobs(z, None, top=top).top_id.cpu().numpy()
    want = R.top_ref(to64(z[:3]), top)
    assert np.array_equal(got[:3], want)
    assert np.array_equal(got[3:], np.broadcast_to(want[0], got[3:].shape))


SIGNALING = {BF16: (torch.int16, 0x7F81), FP16: (torch.int16, 0x7C01),
             FP32: (torch.int32, 0x7F800001)}


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("V,rows", [(3000, 4), (20000, 4), (20000, 515), (140001, 4)])
def test_signaling_nan_among_the_best(V, rows, dt):
    """Any NaN ranks with -inf; the entries around it keep their order."""
    top = 12
    z = logits(rows, V, dt, seed=53)
    itype, bits = SIGNALING[dt]
    i = torch.arange(0, V - 16, V // 9, device=z.device) // 8 * 8
    for e in range(8):   # the best entries beside a NaN, in every place of a chunk
        z[0, i[e] + torch.arange(8, device=z.device)] = 20.0 + e
        z.view(itype)[0, i[e] + e] = bits
        z.view(itype)[2, i[e] + (e + 3) % 8] = bits
        z[2, i[e] + e] = 30.0 - e
    note(f"signaling nan V={V} rows={rows} {dt}")
    ids = swg.token_logprobs(z, None, top=top).top_id[:4].cpu().numpy()
    assert np.array_equal(ids, R.top_ref(to64(z[:4]), top))


# ------------------------------------------------------------------ gradients from the fp32 lse
@pytest.mark.parametrize("dt", [BF16, FP32])
@pytest.mark.parametrize("T", [1e-9, 0.1, 0.7, 1.0])
@pytest.mark.parametrize("V,rows", [(700, 6), (20000, 6), (70001, 6)])
def test_gradients_stay_bounded(V, rows, dt, T):
    """Beside a large |a| the fp32 lse has no room for log sum exp (a - max a): a probability
    may be off, but it stays in [0, 1] and the gradients with it."""
    note(f"bounded gradients T={T} V={V} {dt}")
    z = logits(rows, V, dt, seed=51)
    z[1] = -1e10
    z[2] = -1e20
    z[3] = 3e9
    z[4] = z[4] * 1e8
    t = torch.arange(rows, device=z.device)
    r = swg.token_logprobs(z, t, temperature=T)
    g = torch.ones(rows, device=z.device)
    one = 1.0 + 2 * torch.finfo(dt).eps
    # -p / T away from the target, (1 - p) / T at it
    dz = swg.token_logprobs_bwd(z, t, r.lse, None, g, None, temperature=T).double() * T
    at = torch.zeros(rows, V, dtype=torch.bool, device=z.device)
    at[t, t] = True
    assert float(dz[~at].max()) <= 0 and float(dz[~at].min()) >= -one
    assert float(dz[at].min()) >= 0 and float(dz[at].max()) <= one
    # -p (log p + H) / T with log p <= 0 and p (-log p) <= 1 / e
    de = swg.token_logprobs_bwd(z, None, r.lse, r.entropy, None, g, temperature=T).double() * T
    assert float(de.abs().max()) <= (math.log(V) + 1.0) * one
    u = torch.zeros(rows, 1, device=z.device)
    c = torch.full((rows,), 1.0 / T, device=z.device)
    d = swg.distill_bwd(z, u, t[:, None].contiguous(), r.lse, c, temperature=T).double()
    assert float(d[~at].min()) >= 0 and float(d.abs().max()) <= one


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("V", [40, 5000])
def test_nan_logits_keep_their_gradient_nan(V, dt):
    """A NaN logit beside a finite lse, and a NaN lse beside finite logits."""
    z = logits(2, V, dt, seed=52)
    t = torch.tensor([0, 1], device=z.device)
    r = swg.token_logprobs(z, t)
    at = [1, 9, V - 1]
    z[0, at] = math.nan
    lse = r.lse.clone()
    lse[1] = math.nan
    g = torch.ones(2, device=z.device)
    u = torch.zeros(2, 1, device=z.device)
    for dz in (swg.token_logprobs_bwd(z, t, lse, None, g, None),
               swg.token_logprobs_bwd(z, None, lse, r.entropy, None, g),
               swg.distill_bwd(z, u, t[:, None].contiguous(), lse, g)):
        bad = torch.isnan(dz)
        assert bad[0].nonzero()[:, 0].tolist() == at and bool(bad[1].all())


# ------------------------------------------------------------------ the teacher's range
@pytest.mark.parametrize("udt", DTYPES)
@pytest.mark.parametrize("T", [0.5, 1.0, 4.0])
@pytest.mark.parametrize("V", [500, 40000, 140000])
def test_teacher_values_far_from_zero(V, T, udt):
    """Entries of the type's lowest value (all, some) and its largest, and large values whose
    differences count: q goes by the differences."""
    rows, k = 6, 5
    z = logits(rows, V, BF16, seed=54)
    u, ids = teacher(rows, V, k, udt, pads=False)
    ids[:] = torch.arange(k, device=z.device) * 7
    info = torch.finfo(udt)
    u[0] = info.min
    u[1, 2:] = info.min
    u[2] = info.max
    u[3] = torch.tensor([4096.0, 4096, 4064, 4064, 4032], device=z.device).to(udt) * (
        1 if udt == FP16 else 256)
    u[4] = -u[3]
    c = torch.rand(rows, device=z.device) + 0.5
    note(f"teacher range V={V} T={T} {udt}")
    loss, lse = swg.distill_fwd(z, u, ids, temperature=T)
    check_loss(z, u, ids, T, loss, lse)
    both = swg.distill_fwd_bwd(z, u, ids, c, temperature=T)
    check_loss(z, u, ids, T, both[0], both[1], c, both[2])
    dz = swg.distill_bwd(z, u, ids, lse, c, temperature=T)
    # the same gradient to within the roundings of p from lse (|a| and lse below 64) and of dz
    a, b = dz.double(), both[2].double()
    step = torch.finfo(BF16).eps
    assert bool(((a - b).abs() <= step * b.abs() + 512 * U * c[:, None] * T).all())
