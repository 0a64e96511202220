"""Layer norm, forward and backward, against the float64 oracle."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle.ref as R
import swish_activation_backward_amd as swg
from gpu_util import Guarded, device, note
from parity import to64
from row_models import check, norm_bwd_models, norm_models

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
TYPES = [(BF16, BF16), (BF16, FP32), (FP16, FP16), (FP16, FP32), (FP32, FP32)]
# one element, one lane, one wave, rows around the powers of two that a workgroup's vectors
# end at, odd widths, and rows longer than a workgroup's registers
SHAPES = [(1, 1), (3, 2), (5, 7), (4, 64), (33, 65), (1, 512), (130, 512), (17, 513), (9, 1023),
          (70, 1024), (6, 2047), (5, 2049), (1, 4096), (11, 4097), (3, 8192), (3, 8200),
          (2, 16384), (2, 16387), (2, 40001), (1, 70000)]
EPS = 1e-5


def make(M, N, dt, wdt, seed=0, pad=0, shift=0, scale=1.0, mean=0.5):
    g = torch.Generator().manual_seed(1000 * seed + M + 7 * N)
    dev = device()

    def rows(s):
        buf = torch.full((M * (N + pad) + shift + 8,), float("nan"), dtype=dt, device=dev)
        v = buf[shift:shift + M * (N + pad)].view(M, N + pad)[:, :N]
        v.copy_((torch.randn(M, N, generator=g) * s).to(dt))
        return v

    x = rows(scale)
    x += (mean * torch.randn(M, 1, generator=g)).to(dt).to(dev)
    dy = rows(0.5)
    w = (1 + 0.3 * torch.randn(N, generator=g)).to(wdt).to(dev)
    b = (0.2 * torch.randn(N, generator=g)).to(wdt).to(dev)
    return x, dy, w, b


def check_fwd(x, w, b, y, mean, rstd, eps=EPS):
    ry, rm, rr = R.layer_norm_ref(to64(x), None if w is None else to64(w),
                                  None if b is None else to64(b), float(np.float32(eps)))
    ey, em, er = norm_models(x, w, rm, rr)
    check("mean", mean, rm, em)
    check("rstd", rstd, rr, er)
    if b is not None:
        ey = ey + 2.0 ** -24 * np.abs(to64(b))
    check("y", y, ry, ey)


def check_bwd(dy, x, w, mean, rstd, dx, dw, db, dw0=None, db0=None):
    rdx, rdw, rdb = R.layer_norm_bwd_ref(to64(dy), to64(x), None if w is None else to64(w),
                                         to64(mean), to64(rstd))
    edx, edw, edb = norm_bwd_models(dy, x, w, mean, rstd, dw0, db0)
    if dx is not None:
        check("dx", dx, rdx, edx)
    if dw is not None:
        check("dw", dw, rdw + (0 if dw0 is None else to64(dw0)), edw)
    if db is not None:
        check("db", db, rdb + (0 if db0 is None else to64(db0)), edb)


@pytest.mark.parametrize("dt,wdt", TYPES)
@pytest.mark.parametrize("M,N", SHAPES)
def test_forward_backward(M, N, dt, wdt):
    note(f"layer norm M={M} N={N} {dt} {wdt}")
    x, dy, w, b = make(M, N, dt, wdt)
    dev = x.device
    y = Guarded((M, N), dt, dev)
    mean, rstd = Guarded((M,), FP32, dev), Guarded((M,), FP32, dev)
    dx, dw, db = Guarded((M, N), dt, dev), Guarded((N,), wdt, dev), Guarded((N,), wdt, dev)
    swg.layer_norm_fwd(x, w, b, y.t, mean.t, rstd.t, eps=EPS)
    swg.layer_norm_bwd(dy, x, w, mean.t, rstd.t, dx.t, dw.t, db.t)
    torch.cuda.synchronize()
    check_fwd(x, w, b, y.t, mean.t, rstd.t)
    check_bwd(dy, x, w, mean.t, rstd.t, dx.t, dw.t, db.t)
    for o in (y, mean, rstd, dx, dw, db):
        o.check()


@pytest.mark.parametrize("M,N", [(1500, 512), (5000, 96), (20011, 33), (700, 4096), (300, 16384),
                                 (129, 20000)])
@pytest.mark.parametrize("dt,wdt", [(BF16, FP32), (FP32, FP32)])
def test_many_rows(M, N, dt, wdt):
    note(f"layer norm many rows M={M} N={N} {dt}")
    x, dy, w, b = make(M, N, dt, wdt, seed=1)
    y, mean, rstd = swg.layer_norm_fwd(x, w, b, eps=EPS)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
    swg.layer_norm_bwd(dy, x, w, mean, rstd, dx, dw, db)
    check_fwd(x, w, b, y, mean, rstd)
    check_bwd(dy, x, w, mean, rstd, dx, dw, db)
    # no run-to-run change
    dx2, dw2, db2 = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
    swg.layer_norm_bwd(dy, x, w, mean, rstd, dx2, dw2, db2)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2) and torch.equal(db, db2)


@pytest.mark.parametrize("dt", [BF16, FP16, FP32])
@pytest.mark.parametrize("N,pad,shift", [(512, 8, 0), (512, 1, 0), (511, 2, 3), (1000, 24, 1),
                                         (4097, 3, 5), (64, 64, 7), (17000, 1, 1)])
def test_row_strides_and_alignment(N, pad, shift, dt):
    """Rows inside wider buffers, first elements on any element boundary; the elements
    between the rows (NaN here) are neither read nor written."""
    M = 13
    note(f"layer norm strided N={N} pad={pad} shift={shift} {dt}")
    x, dy, w, b = make(M, N, dt, dt, seed=2, pad=pad, shift=shift)
    dev = x.device
    yb = torch.full((M, N + pad), 7.0, dtype=dt, device=dev)
    dxb = torch.full((M, N + pad), 7.0, dtype=dt, device=dev)
    y, dx = yb[:, :N], dxb[:, :N]
    y, mean, rstd = swg.layer_norm_fwd(x, w, b, y, eps=EPS)
    dw, db = torch.empty_like(w), torch.empty_like(b)
    swg.layer_norm_bwd(dy, x, w, mean, rstd, dx, dw, db)
    check_fwd(x, w, b, y, mean, rstd)
    check_bwd(dy, x, w, mean, rstd, dx, dw, db)
    assert bool((yb[:, N:] == 7).all()) and bool((dxb[:, N:] == 7).all())


@pytest.mark.parametrize("N", [96, 5000, 17000])
def test_optional_operands(N):
    M = 37
    x, dy, w, b = make(M, N, BF16, FP32, seed=3)
    for ww, bb in ((None, None), (w, None), (None, b)):
        y, mean, rstd = swg.layer_norm_fwd(x, ww, bb, eps=EPS)
        check_fwd(x, ww, bb, y, mean, rstd)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
    for odx, odw, odb in ((dx, None, None), (None, dw, db), (dx, dw, None), (dx, None, db),
                          (None, None, None)):
        for ww in (w, None):
            for o in (dx, dw, db):
                o.fill_(7.0)
            swg.layer_norm_bwd(dy, x, ww, mean, rstd, odx, odw, odb)
            check_bwd(dy, x, ww, mean, rstd, odx, odw, odb)
            for o, want in ((dx, odx), (dw, odw), (db, odb)):
                assert want is not None or bool((o == 7).all())


@pytest.mark.parametrize("wdt", [BF16, FP32])
@pytest.mark.parametrize("M", [0, 1, 300])
def test_accumulate(M, wdt):
    N = 200
    x, dy, w, b = make(M, N, BF16, wdt, seed=4)
    mean, rstd = (torch.empty(M, device=x.device) for _ in range(2))
    swg.layer_norm_fwd(x, w, b, None, mean, rstd, eps=EPS)
    dw0, db0 = torch.randn(2, N, device=x.device).to(wdt)
    dw, db = dw0.clone(), db0.clone()
    dx = torch.empty_like(x)
    swg.layer_norm_bwd(dy, x, w, mean, rstd, dx, dw, db, accumulate=True)
    if M == 0:
        assert torch.equal(dw, dw0) and torch.equal(db, db0)
        swg.layer_norm_bwd(dy, x, w, mean, rstd, dx, dw, db)
        assert not dw.any() and not db.any()
        return
    check_bwd(dy, x, w, mean, rstd, dx, dw, db, dw0, db0)


@pytest.mark.parametrize("N", [64, 777, 4096, 20000])
def test_values_where_norms_go_wrong(N):
    """Constant rows (variance 0), a mean far above the spread, tiny and huge values, and rows
    with NaN or infinities beside ordinary ones."""
    x, dy, w, b = make(8, N, FP32, FP32, seed=5)
    x[0] = 3.0
    x[1] = 0.0
    x[2] += 1000.0
    x[3] *= 1e-12
    x[4] *= 1e15
    x[5, N // 2] = float("nan")
    x[6, N // 3] = float("inf")
    y, mean, rstd = swg.layer_norm_fwd(x, w, b, eps=EPS)
    ok = [0, 1, 2, 3, 4, 7]
    check_fwd(x[ok], w, b, y[ok], mean[ok], rstd[ok])
    assert bool(torch.isnan(y[5]).all()) and bool(torch.isnan(y[6]).any())
    dx = torch.empty_like(x)
    swg.layer_norm_bwd(dy, x, w, mean, rstd, dx, None, None)
    check_bwd(dy[ok], x[ok], w, mean[ok], rstd[ok], dx[ok], None, None)
    assert bool(torch.isnan(dx[5]).all())


def test_offsets_past_32_bits():
    """Rows more than 2^31 elements apart."""
    dev = device()
    N, ld = 1000, (1 << 31) // 2 + 24
    buf = torch.empty(2 * ld + N, dtype=BF16, device=dev)
    x = torch.as_strided(buf, (3, N), (ld, 1))
    src, dy, w, b = make(3, N, BF16, BF16, seed=6)
    x.copy_(src)
    assert x[2].data_ptr() - x.data_ptr() >= 1 << 32
    y, mean, rstd = swg.layer_norm_fwd(x, w, b, eps=EPS)
    check_fwd(src, w, b, y, mean, rstd)
    dw, db = torch.empty_like(w), torch.empty_like(b)
    dx = torch.empty_like(src)
    swg.layer_norm_bwd(dy, x, w, mean, rstd, dx, dw, db)
    check_bwd(dy, src, w, mean, rstd, dx, dw, db)


def test_other_stream_and_graph():
    """On a stream of its own, and captured into a graph that replays with new inputs."""
    M, N = 700, 520
    x, dy, w, b = make(M, N, BF16, BF16, seed=7)
    y, mean, rstd = swg.layer_norm_fwd(x, w, b, eps=EPS)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
    ws = torch.empty(swg.layer_norm_bwd_workspace_size(M, N, BF16), dtype=torch.uint8,
                     device=x.device)

    def step(stream=None):
        swg.layer_norm_fwd(x, w, b, y, mean, rstd, eps=EPS, stream=stream)
        swg.layer_norm_bwd(dy, x, w, mean, rstd, dx, dw, db, workspace=ws, stream=stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    torch.cuda.current_stream().wait_stream(side)
    check_fwd(x, w, b, y, mean, rstd)
    check_bwd(dy, x, w, mean, rstd, dx, dw, db)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        x2, dy2, _, _ = make(M, N, BF16, BF16, seed=20 + i)
        x.copy_(x2)
        dy.copy_(dy2)
        for o in (y, dx, dw, db):
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (y, mean, rstd, dx, dw, db)]
        step()
        torch.cuda.synchronize()
        for a, c in zip(got, (y, mean, rstd, dx, dw, db)):
            assert torch.equal(a, c)


@pytest.mark.parametrize("N", [5, 24])
def test_more_rows_than_workgroups(N):
    """More than 2^20 rows, repeating with an odd period."""
    period, M = 1009, (1 << 20) + 5000
    note(f"layer norm rows {M} N={N}")
    x1, dy1, w, b = make(period, N, BF16, FP32, seed=8)
    i = torch.arange(M, device=x1.device) % period
    x, dy = x1[i], dy1[i]
    y1, m1, r1 = swg.layer_norm_fwd(x1, w, b, eps=EPS)
    check_fwd(x1, w, b, y1, m1, r1)
    y, m, r = swg.layer_norm_fwd(x, w, b, eps=EPS)
    assert torch.equal(y, y1[i]) and torch.equal(m, m1[i]) and torch.equal(r, r1[i])
    dx1, dx = torch.empty_like(x1), torch.empty_like(x)
    dw, db = torch.empty_like(w), torch.empty_like(b)
    swg.layer_norm_bwd(dy1, x1, w, m1, r1, dx1, None, None)
    check_bwd(dy1, x1, w, m1, r1, dx1, None, None)
    swg.layer_norm_bwd(dy, x, w, m, r, dx, dw, db)
    assert torch.equal(dx, dx1[i])
    check_bwd(dy, x, w, m, r, None, dw, db)
