"""The linear layer and the residual norm on other streams, in replayed graphs, at both tiles, over
shapes whose tiles are whole rounds and a rest, and beyond 32-bit offsets."""
from __future__ import annotations

import pytest
import torch

import swish_activation_backward_amd as swg
from gpu_util import device, note

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


def rnd(g, *s, dt=BF16, scale=1.0):
    return (torch.randn(*s, device="cuda", generator=g) * scale).to(dt)


def sum_bound(dt, mag):
    """Half a step of the type on top of fp32 sums' 2^-16 of the magnitude sum."""
    return lambda ref: torch.finfo(dt).eps / 2 * ref.abs() + 2.0 ** -16 * mag + 1e-30


@pytest.fixture
def gen():
    device()
    return torch.Generator(device="cuda").manual_seed(11)


@pytest.fixture
def tile():
    yield swg.swg_set_gemm_tile
    swg.swg_set_gemm_tile(0)


@pytest.mark.parametrize("nk", [False, True], ids=["kn", "nk"])
@pytest.mark.parametrize("M,K,N", [(700, 328, 520), (90, 2000, 264), (260, 64, 1000)])
@pytest.mark.parametrize("edge", [256, 128])
def test_both_tiles(gen, tile, edge, M, K, N, nk):
    note(f"linear tile {edge} M={M} K={K} N={N} nk={nk}")
    tile(edge)
    x, w = rnd(gen, M, K), rnd(gen, N, K, scale=K ** -0.5).t() if nk else rnd(gen, K, N,
                                                                             scale=K ** -0.5)
    dy, res, b = rnd(gen, M, N), rnd(gen, M, N), rnd(gen, N)
    y = swg.linear_fwd(x, w, b, res)
    dx = torch.empty_like(x)
    dw = torch.empty(N, K, dtype=BF16, device="cuda").t() if nk else torch.empty_like(w)
    swg.linear_bwd(dy, x, w, None, dx, dw)
    torch.cuda.synchronize()
    xd, wd, dyd = x.double(), w.double(), dy.double()
    for got, ref, mag in ((y, xd @ wd + b.double() + res.double(),
                           xd.abs() @ wd.abs() + b.double().abs() + res.double().abs()),
                          (dx, dyd @ wd.t(), dyd.abs() @ wd.abs().t()),
                          (dw, xd.t() @ dyd, xd.abs().t() @ dyd.abs())):
        assert ((got.double() - ref).abs() <= sum_bound(BF16, mag)(ref)).all()


def test_tile_setting_between_calls_of_one_shape(gen, tile):
    """The workspace a call allocates is the one of its tile."""
    x, w = rnd(gen, 130, 4096), rnd(gen, 4096, 136, scale=1 / 64)
    ref = x.double() @ w.double()
    for edge in (0, 128, 256, 128, 0):
        tile(edge)
        y = swg.linear_fwd(x, w)
        torch.cuda.synchronize()
        bound = sum_bound(BF16, x.double().abs() @ w.double().abs())(ref)
        assert ((y.double() - ref).abs() <= bound).all(), edge


# tiles of 256: 17 x 16 (one whole round and 16 left, split), 33 x 17; fp32: 64-tiles
@pytest.mark.parametrize("M,K,N,dt", [(4350, 1032, 4096, BF16), (8200, 2056, 4304, FP16),
                                      (2080, 1000, 2052, FP32)])
def test_whole_rounds_and_a_rest(gen, M, K, N, dt):
    note(f"linear M={M} K={K} N={N} {dt}")
    x, w, res = rnd(gen, M, K, dt=dt), rnd(gen, K, N, dt=dt, scale=K ** -0.5), rnd(gen, M, N, dt=dt)
    bias = rnd(gen, N, dt=dt)
    z = torch.empty(M, N, dtype=dt, device="cuda")
    y = swg.linear_fwd(x, w, bias, res, "relu", z=z)
    torch.cuda.synchronize()
    zd = x.double() @ w.double() + bias.double()
    mag = x.double().abs() @ w.double().abs() + bias.double().abs()
    assert ((z.double() - zd).abs() <= sum_bound(dt, mag)(zd)).all()
    yd = zd.relu() + res.double()
    assert ((y.double() - yd).abs() <= sum_bound(dt, mag + res.double().abs())(yd)).all()


def calls(gen):
    """Name -> call of no arguments that returns its outputs; the sizes take every launch."""
    out = {}

    def linear(M, K, N, dt, act, nk=False):
        x, res, dy = rnd(gen, M, K, dt=dt), rnd(gen, M, N, dt=dt), rnd(gen, M, N, dt=dt)
        w = rnd(gen, N, K, dt=dt, scale=K ** -0.5).t() if nk else rnd(gen, K, N, dt=dt,
                                                                     scale=K ** -0.5)
        b, z = rnd(gen, N, dt=dt), torch.empty(M, N, dtype=dt, device="cuda")
        y, dx, db = torch.empty_like(res), torch.empty_like(x), torch.empty_like(b)
        dw = torch.empty(w.t().shape if nk else w.shape, dtype=dt, device="cuda")
        dw = dw.t() if nk else dw
        rows16 = K % 8 == 0 and N % 8 == 0
        ws = torch.empty(max(swg.linear_fwd_workspace_size(M, K, N, dt, nk, rows16),
                             swg.linear_bwd_workspace_size(M, K, N, dt, act, nk, rows16), 1),
                         dtype=torch.uint8, device="cuda")

        def run(stream=None):
            swg.linear_fwd(x, w, b, res, act, y=y, z=z, workspace=ws, stream=stream)
            swg.linear_bwd(dy, x, w, z, dx, dw, db, act, workspace=ws, stream=stream)
            return y, z, dx, dw, db
        return run

    def norm(M, N, gate):
        y, res, dout, dn = (rnd(gen, M, N) for _ in range(4))
        wp, wq, dwp, dwq = (rnd(gen, N) for _ in range(4))
        gv = {"channel": lambda: rnd(gen, N), "row": lambda: rnd(gen, M, 1),
              "full": lambda: rnd(gen, M, N)}[gate]()
        rs, rp = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
        o, n, dy, dr, dg = (torch.empty_like(t) for t in (y, y, y, y, gv))
        ws = torch.empty(swg.residual_norm_bwd_workspace_size(M, N, BF16), dtype=torch.uint8,
                         device="cuda")

        def run(stream=None):
            swg.residual_norm_fwd(y, res, wp, wq, gv, 0.5, out=o, norm=n, stats=True, rstd_post=rs,
                                  rstd_pre=rp, stream=stream)
            swg.residual_norm_bwd(dout, dn, y, o, wp, wq, gv, rs, rp, dy, dr, dwp, dwq, dg, 0.5,
                                  workspace=ws, stream=stream)
            return o, n, rs, rp, dy, dr, dwp, dwq, dg
        return run

    out["split"] = linear(40, 3000, 264, BF16, "gelu")
    out["packed"] = linear(150, 203, 77, FP16, "swish", nk=True)
    out["tiles"] = linear(1500, 256, 512, BF16, "none")
    out["fp32"] = linear(70, 600, 130, FP32, "gelu_tanh")
    out["norm"] = norm(500, 768, "channel")
    out["norm row"] = norm(33, 5000, "row")
    out["norm long"] = norm(9, 20001, "full")
    return out


def test_graph_replays(gen):
    """Captured calls, replayed with other work and synchronisations between, give the eager bits
    for the inputs of each replay."""
    for name, run in calls(gen).items():
        note(f"graph {name}")
        run()
        torch.cuda.synchronize()
        want = [t.clone() for t in run()]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = run()
        for _ in range(4):
            for t in outs:
                t.fill_(float("nan"))
            torch.randn(1000, 1000, device="cuda") @ torch.randn(1000, 1000, device="cuda")
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(outs, want)), name


def test_streams_and_two_calls_at_once(gen):
    """A given stream, a current stream, and calls on two streams at once with own workspaces."""
    runs = calls(gen)
    want = {}
    for n, run in runs.items():
        want[n] = [t.clone() for t in run()]
    torch.cuda.synchronize()
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = {}
    for i, (n, run) in enumerate(runs.items()):
        s = side[i % 2]
        if i % 3 == 0:
            with torch.cuda.stream(s):
                got[n] = run()
        else:
            got[n] = run(stream=s)
    torch.cuda.synchronize()
    for n in runs:
        assert all(torch.equal(a, b) for a, b in zip(got[n], want[n])), n


def test_linear_beyond_32_bit_offsets(gen):
    """More than 2^32 bytes of x and of y: the last rows equal those of a small call."""
    M, K, N = (1 << 20) + 70, 2056, 8
    note(f"linear M={M} K={K} N={N}")
    x = torch.zeros(M, K, dtype=BF16, device="cuda")
    x[-300:] = rnd(gen, 300, K)
    w = rnd(gen, K, N, scale=K ** -0.5)
    y = swg.linear_fwd(x, w)
    tail = swg.linear_fwd(x[-300:].clone(), w)
    torch.cuda.synchronize()
    ref = x[-300:].double() @ w.double()
    mag = x[-300:].double().abs() @ w.double().abs()
    for t in (y[-300:], tail):
        assert ((t.double() - ref).abs() <= sum_bound(BF16, mag)(ref)).all()
    assert not y[:-300].any()
    del x, y
    wide = swg.linear_fwd(rnd(gen, (1 << 16) + 5, 16), rnd(gen, 16, 1 << 15) * 0 + 1)   # y > 2^32 B
    torch.cuda.synchronize()
    # every column is the same sum
    assert torch.equal(wide[-7:, 0], wide[-7:, -1]) and torch.equal(wide[:, 1], wide[:, -2])


def test_residual_norm_beyond_32_bit_offsets(gen):
    M, N = (1 << 19) + 9, 4224
    note(f"residual norm M={M} N={N}")
    y = torch.empty(M, N, dtype=BF16, device="cuda")
    y[:-64] = 1.0
    y[-64:] = rnd(gen, 64, N)
    w = rnd(gen, N)
    r = swg.residual_norm_fwd(y, None, w, w, stats=True)
    small = swg.residual_norm_fwd(y[-64:].clone(), None, w, w, stats=True)
    dy = torch.empty_like(y)
    swg.residual_norm_bwd(None, y, y, r.out, w, w, None, r.rstd_post, r.rstd_pre, dy, None)
    dsmall = torch.empty(64, N, dtype=BF16, device="cuda")
    swg.residual_norm_bwd(None, y[-64:].clone(), y[-64:].clone(), small.out, w, w, None,
                          small.rstd_post, small.rstd_pre, dsmall, None)
    torch.cuda.synchronize()
    for a, b in zip(r, small):
        assert torch.equal(a[-64:], b)
    assert torch.equal(dy[-64:], dsmall)


def test_linear_rows_far_apart(gen):
    """Strides that the tiles' windows do not reach: the operands are laid out again."""
    far = (1 << 22) + 8
    note(f"linear strides {far}")
    x = torch.zeros(33, far, dtype=BF16, device="cuda")[:, :64]
    x.copy_(rnd(gen, 33, 64))
    w = torch.zeros(64, far, dtype=BF16, device="cuda")[:, :72]
    w.copy_(rnd(gen, 64, 72, scale=0.1))
    dy = torch.zeros(33, far, dtype=BF16, device="cuda")[:, :72]
    dy.copy_(rnd(gen, 33, 72))
    y, dx = torch.zeros_like(dy), torch.empty(33, 64, dtype=BF16, device="cuda")
    dw = torch.empty(64, 72, dtype=BF16, device="cuda")
    swg.linear_fwd(x, w, y=y)
    swg.linear_bwd(dy, x, w, None, dx, dw)
    x, w, dy = x.double().cpu(), w.double().cpu(), dy.double().cpu()
    for got, a, b in ((y, x, w), (dx, dy, w.t()), (dw, x.t(), dy)):
        ref, mag = a @ b, a.abs() @ b.abs()
        assert ((got.double().cpu() - ref).abs() <= sum_bound(BF16, mag)(ref)).all()


def test_linear_more_tiles_than_a_launch(gen):
    """fp32 tiles of 2^30 rows are launched in parts."""
    M = (1 << 30) + 70
    note(f"linear M={M} K=4 N=4 fp32")
    w = rnd(gen, 4, 4, dt=FP32)
    x = torch.empty(M, 4, dtype=FP32, device="cuda")
    line = rnd(gen, 4099, 4, dt=FP32)
    for r in range(0, M, 4099 * 4096):
        part = x[r:r + 4099 * 4096]
        part.copy_(line.repeat(4096, 1)[:part.shape[0]])
    y = swg.linear_fwd(x, w)
    want = swg.linear_fwd(line, w)
    ref = line.double() @ w.double()
    mag = line.double().abs() @ w.double().abs()
    assert ((want.double() - ref).abs() <= sum_bound(FP32, mag)(ref)).all()
    for r in range(0, M, 4099 * 4096):
        part = y[r:r + 4099 * 4096]
        assert torch.equal(part, want.repeat(4096, 1)[:part.shape[0]]), r
