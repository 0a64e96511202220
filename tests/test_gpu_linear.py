"""Linear layer with its epilogue, forward and backward, against the float64 oracle."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle.ref as R
import swish_activation_backward_amd as swg
from gpu_util import Guarded, device, note
from linear_models import bwd_models, fwd_models
from parity import to64
from row_models import check

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
TYPES = [BF16, FP16, FP32]
ACTS = ["none", "relu", "swish", "gelu", "gelu_tanh"]
# single tokens, the edges of the few-token form, of the tiles and of the contraction's stages,
# sizes that divide by nothing, and contractions long enough to be split
SHAPES = [(1, 1, 1), (1, 64, 64), (1, 4096, 512), (2, 9, 5), (3, 1000, 1001), (5, 1023, 77),
          (16, 256, 384), (17, 520, 264), (33, 136, 128), (64, 512, 1024), (64, 130, 96),
          (65, 96, 72), (100, 333, 257), (128, 256, 256), (200, 64, 1030), (257, 1024, 520),
          (300, 8, 8), (513, 200, 300), (1030, 160, 136), (700, 2056, 24), (40, 6000, 200),
          (130, 5000, 130)]


def make(M, K, N, dt, nk=False, seed=0, pad=0, shift=0, res_scale=1.0):
    g = torch.Generator().manual_seed(1000 * seed + M + 7 * K + 13 * N)
    dev = device()

    def rows(r, c, s=1.0):
        buf = torch.full((r * (c + pad) + shift + 8,), float("nan"), dtype=dt, device=dev)
        v = buf[shift:shift + r * (c + pad)].view(r, c + pad)[:, :c]
        v.copy_((torch.randn(r, c, generator=g) * s).to(dt))
        return v

    s = max(K, 1) ** -0.5
    d = {"x": rows(M, K), "w": rows(N, K, s).t() if nk else rows(K, N, s),
         "residual": rows(M, N, res_scale), "dy": rows(M, N, 0.5), "z": rows(M, N, 1.5)}
    d["bias"] = (0.3 * torch.randn(N, generator=g)).to(dt).to(dev)
    return d


def f64(t):
    return None if t is None else to64(t)


def check_fwd(d, y, z, act="none", beta=1.0, bias=True, residual=True):
    b, r = d["bias"] if bias else None, d["residual"] if residual else None
    ry, rz = R.linear_ref(to64(d["x"]), to64(d["w"]), f64(b), f64(r), act,
                          float(np.float32(beta)))
    ey, ez = fwd_models(d["x"], d["w"], b, r, act, ry, rz)
    check("y", y, ry, ey)
    if z is not None:
        check("z", z, rz, ez)


def check_bwd(d, dx, dw, db, act="none", beta=1.0, init=None):
    rdx, rdw, rdb, dz = R.linear_bwd_ref(to64(d["dy"]), to64(d["x"]), to64(d["w"]), to64(d["z"]),
                                         act, float(np.float32(beta)))
    edx, edw, edb = bwd_models(d["dy"], d["x"], d["w"], d["z"], act, dz)
    if dx is not None:
        check("dx", dx, rdx, edx)
    for name, got, ref, e in (("dw", dw, rdw, edw), ("db", db, rdb, edb)):
        if got is None:
            continue
        if init:
            ref, e = ref + to64(init[name]), e + 2.0 ** -24 * np.abs(to64(init[name]))
        check(name, got, ref, e)


def run_both(d, M, K, N, dt, nk, act, beta=1.0, bias=True, residual=True, keep=True):
    dev, bands = d["x"].device, []

    def new(*shape):
        bands.append(Guarded(shape, dt, dev))
        return bands[-1].t

    y, z = new(M, N), new(M, N) if keep else None
    got = swg.linear_fwd(d["x"], d["w"], d["bias"] if bias else None,
                         d["residual"] if residual else None, act, beta, y=y, z=z)
    assert got is y
    dx, dw, db = new(M, K), new(N, K).t() if nk else new(K, N), new(N)
    swg.linear_bwd(d["dy"], d["x"], d["w"], d["z"], dx, dw, db, act, beta)
    torch.cuda.synchronize()
    check_fwd(d, y, z, act, beta, bias, residual)
    check_bwd(d, dx, dw, db, act, beta)
    for b in bands:
        b.check()


@pytest.mark.parametrize("nk", [False, True], ids=["kn", "nk"])
@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_shapes_types_layouts(M, K, N, dt, nk):
    i = M + K + N + nk
    act = ACTS[i % 5]
    note(f"linear M={M} K={K} N={N} {dt} nk={nk} {act}")
    run_both(make(M, K, N, dt, nk), M, K, N, dt, nk, act, bias=i % 2 == 0, residual=i % 3 != 0,
             keep=i % 4 != 0)


# few rows whose weight has its contraction contiguous (K forward of [N, K], N backward of [K, N]):
# the ends of a lane's 16 bytes, of a step, of a wave's run and of a turn of all waves
@pytest.mark.parametrize("nk", [False, True], ids=["kn", "nk"])
@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("deep", [1, 7, 8, 9, 31, 33, 64, 127, 128, 129, 2047, 2048, 2049, 4225])
@pytest.mark.parametrize("M,other", [(1, 16), (2, 1), (15, 17), (16, 250)])
def test_few_rows(M, other, deep, dt, nk):
    K, N = (deep, other) if nk else (other, deep)
    note(f"linear few rows M={M} K={K} N={N} {dt} nk={nk}")
    i = M + deep
    run_both(make(M, K, N, dt, nk, pad=deep % 3), M, K, N, dt, nk, ACTS[i % 5], bias=i % 2 == 0,
             residual=i % 3 != 0)


# up to 4 rows against a weight in rows: the ends of a lane's 8 rows, of a wave's run and of a turn,
# and of the columns' chunks
@pytest.mark.parametrize("nk", [False, True], ids=["kn", "nk"])
@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("flat", [1, 7, 8, 9, 127, 128, 129, 1921, 2047, 2048, 2049])
@pytest.mark.parametrize("M,other", [(1, 8), (2, 9), (3, 33), (4, 250)])
def test_few_rows_against_rows(M, other, flat, dt, nk):
    K, N = (other, flat) if nk else (flat, other)
    note(f"linear few rows against rows M={M} K={K} N={N} {dt} nk={nk}")
    i = M + flat
    run_both(make(M, K, N, dt, nk, pad=flat % 3), M, K, N, dt, nk, ACTS[i % 5], bias=i % 2 == 0,
             residual=i % 3 != 0)


@pytest.mark.parametrize("act,beta", [(a, 1.0) for a in ACTS] + [("swish", 1.702), ("swish", 0.0),
                                                                 ("swish", -2.0)])
@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("M,K,N", [(3, 72, 40), (150, 40, 136), (40, 24, 600)])
def test_activations(M, K, N, dt, act, beta):
    note(f"linear M={M} K={K} N={N} {dt} {act} {beta}")
    run_both(make(M, K, N, dt, seed=1), M, K, N, dt, False, act, beta)


@pytest.mark.parametrize("nk", [False, True], ids=["kn", "nk"])
@pytest.mark.parametrize("pad,shift", [(8, 0), (1, 0), (3, 1), (16, 4)])
@pytest.mark.parametrize("dt", [BF16, FP32])
@pytest.mark.parametrize("M,K,N", [(7, 96, 160), (150, 200, 264), (70, 33, 47)])
def test_strides_and_alignment(M, K, N, dt, pad, shift, nk):
    note(f"linear M={M} K={K} N={N} {dt} pad={pad} shift={shift} nk={nk}")
    run_both(make(M, K, N, dt, nk, seed=2, pad=pad, shift=shift), M, K, N, dt, nk, "swish")


@pytest.mark.parametrize("pad", [8, 5])
@pytest.mark.parametrize("M,K,N", [(4, 64, 72), (140, 64, 136)])
def test_strided_outputs(M, K, N, pad):
    """Outputs inside wider buffers; what lies between their rows stays."""
    d = make(M, K, N, BF16, seed=3)
    wide = {n: torch.full((r, c + pad), 7.0, dtype=BF16, device=d["x"].device)
            for n, r, c in (("y", M, N), ("z", M, N), ("dx", M, K), ("dw", K, N))}
    v = {n: t[:, :-pad] for n, t in wide.items()}
    swg.linear_fwd(d["x"], d["w"], d["bias"], d["residual"], "gelu", y=v["y"], z=v["z"])
    swg.linear_bwd(d["dy"], d["x"], d["w"], d["z"], v["dx"], v["dw"], None, "gelu")
    torch.cuda.synchronize()
    check_fwd(d, v["y"], v["z"], "gelu")
    check_bwd(d, v["dx"], v["dw"], None, "gelu")
    assert all((t[:, -pad:] == 7.0).all() for t in wide.values())


@pytest.mark.parametrize("M,K,N", [(1, 512, 256), (9, 100, 51), (130, 72, 264), (300, 3000, 40)])
@pytest.mark.parametrize("dt", TYPES)
def test_residual_in_place(M, K, N, dt):
    d = make(M, K, N, dt, seed=4)
    want = swg.linear_fwd(d["x"], d["w"], d["bias"], d["residual"], "relu")
    y = d["residual"].clone()
    assert swg.linear_fwd(d["x"], d["w"], d["bias"], y, "relu", y=y) is y
    torch.cuda.synchronize()
    assert torch.equal(y, want)


@pytest.mark.parametrize("nk", [False, True], ids=["kn", "nk"])
@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("M,K,N", [(5, 40, 48), (300, 136, 72), (2000, 64, 65)])
def test_accumulate(M, K, N, dt, nk):
    d = make(M, K, N, dt, nk, seed=5)
    dev = d["x"].device
    init = {"dw": torch.randn(K, N, device=dev).to(dt), "db": torch.randn(N, device=dev).to(dt)}
    for accumulate in (False, True):
        dw = init["dw"].t().contiguous().t() if nk else init["dw"].clone()
        db = init["db"].clone()
        swg.linear_bwd(d["dy"], d["x"], d["w"], d["z"], None, dw, db, "gelu_tanh",
                       accumulate=accumulate)
        torch.cuda.synchronize()
        check_bwd(d, None, dw, db, "gelu_tanh", init=init if accumulate else None)


@pytest.mark.parametrize("act", ["none", "swish"])
@pytest.mark.parametrize("M,K,N", [(3, 40, 24), (150, 130, 70)])
def test_single_gradients(M, K, N, act):
    d = make(M, K, N, BF16, seed=6)
    dev = d["x"].device
    z = None if act == "none" else d["z"]
    new = lambda *s: torch.full(s, float("nan"), dtype=BF16, device=dev)  # noqa: E731
    for want in ("dx", "dw", "db"):
        dx = new(M, K) if want == "dx" else None
        dw = new(K, N) if want == "dw" else None
        db = new(N) if want == "db" else None
        swg.linear_bwd(d["dy"], d["x"] if dw is not None else None,
                       d["w"] if dx is not None else None, z, dx, dw, db, act)
        torch.cuda.synchronize()
        check_bwd(d, dx, dw, db, act)


@pytest.mark.parametrize("dt", TYPES)
def test_empty_sizes(dt):
    dev = device()
    e = lambda *s: torch.empty(*s, dtype=dt, device=dev)  # noqa: E731
    bias, res = torch.randn(24, device=dev).to(dt), torch.randn(5, 24, device=dev).to(dt)
    y = swg.linear_fwd(e(5, 0), e(0, 24), bias, res, "relu")      # the empty sums
    assert torch.equal(y, (bias.float().clamp(min=0) + res.float()).to(dt))
    assert swg.linear_fwd(e(0, 16), e(16, 24)).shape == (0, 24)
    assert swg.linear_fwd(e(5, 16), e(16, 0)).shape == (5, 0)
    one = torch.ones(16, 24, dtype=dt, device=dev)
    dw, db = one.clone(), torch.ones(24, dtype=dt, device=dev)
    swg.linear_bwd(e(0, 24), e(0, 16), one, None, e(0, 16), dw, db, accumulate=True)
    assert (dw == 1).all() and (db == 1).all()
    swg.linear_bwd(e(0, 24), e(0, 16), one, None, e(0, 16), dw, db)
    assert not dw.any() and not db.any()
    dx = torch.ones(5, 16, dtype=dt, device=dev)
    swg.linear_bwd(e(5, 0), e(5, 16), e(16, 0), None, dx, e(16, 0))
    assert not dx.any()


@pytest.mark.parametrize("M,K,N", [(4, 64, 48), (4, 33, 47), (200, 160, 136), (200, 67, 41)])
@pytest.mark.parametrize("dt", TYPES)
def test_special_values_stay_in_their_rows(M, K, N, dt):
    d = make(M, K, N, dt, seed=7)
    want = swg.linear_fwd(d["x"], d["w"], d["bias"], act="relu")
    d["x"][1, K // 2] = float("nan")
    d["x"][3, 0] = float("inf")
    y = swg.linear_fwd(d["x"], d["w"], d["bias"], act="relu")
    torch.cuda.synchronize()
    keep = [i for i in range(M) if i not in (1, 3)]
    assert torch.equal(y[keep], want[keep])
    assert y[1].isnan().all()
    # inf times a weight of either sign, none of them 0
    assert torch.equal(y[3], torch.where(d["w"][0] > 0, float("inf"), 0.0).to(dt))


@pytest.mark.parametrize("M", [3, 50, 500])
def test_repeats_bit_for_bit(M):
    K, N = 2000, 264
    d = make(M, K, N, BF16, seed=8)
    first = None
    for _ in range(3):
        y = swg.linear_fwd(d["x"], d["w"], d["bias"], act="gelu")
        dx, dw = torch.empty_like(d["x"]), torch.empty_like(d["w"])
        db = torch.empty_like(d["bias"])
        swg.linear_bwd(d["dy"], d["x"], d["w"], d["z"], dx, dw, db, "gelu")
        torch.cuda.synchronize()
        now = (y, dx, dw, db)
        first = first or now
        assert all(torch.equal(a, b) for a, b in zip(first, now))
