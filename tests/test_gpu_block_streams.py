"""The linear layer and the residual norm on streams that make their inputs, in graphs replayed on
new inputs, and beyond 32-bit offsets with rows that all differ: a call that runs nothing, late, on
another stream or on other rows gives other bits."""
from __future__ import annotations

import pytest
import torch

import swish_activation_backward_amd as swg
from gpu_util import device, note

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


class Linear:
    """A forward and backward call with own outputs, inputs and (where asked for) workspace."""

    def __init__(self, M, K, N, dt, act, nk=False, own=True):
        dev = device()
        new = lambda *s: torch.empty(*s, dtype=dt, device=dev)  # noqa: E731
        w = new(N, K) if nk else new(K, N)
        dw = torch.empty_like(w)
        self.act, self.scale = act, K ** -0.5
        self.inputs = {"x": new(M, K), "w": w, "b": new(N), "res": new(M, N), "dy": new(M, N)}
        self.w, self.dw = (w.t(), dw.t()) if nk else (w, dw)
        self.y, self.z, self.dx, self.db = new(M, N), new(M, N), new(M, K), new(N)
        self.outputs = [self.y, self.z, self.dx, dw, self.db]
        self.ws = None
        if own:
            rows16 = K % 8 == 0 and N % 8 == 0
            self.ws = torch.empty(max(swg.linear_fwd_workspace_size(M, K, N, dt, nk, rows16),
                                      swg.linear_bwd_workspace_size(M, K, N, dt, act, nk, rows16),
                                      1), dtype=torch.uint8, device=dev)

    def run(self, stream=None):
        i = self.inputs
        swg.linear_fwd(i["x"], self.w, i["b"], i["res"], self.act, y=self.y, z=self.z,
                       workspace=self.ws, stream=stream)
        swg.linear_bwd(i["dy"], i["x"], self.w, self.z, self.dx, self.dw, self.db, self.act,
                       workspace=self.ws, stream=stream)


class Norm:
    scale = 1.0

    def __init__(self, M, N, gate, own=True):
        dev = device()
        new = lambda *s: torch.empty(*s, dtype=BF16, device=dev)  # noqa: E731
        self.inputs = {n: new(M, N) for n in ("y", "res", "dout", "dn")}
        self.inputs.update(wp=new(N), w=new(N),
                           gate=new(*{"channel": (N,), "row": (M, 1), "full": (M, N)}[gate]))
        o, n, dy, dr = (new(M, N) for _ in range(4))
        dwp, dwq, dg = new(N), new(N), torch.empty_like(self.inputs["gate"])
        rs, rp = torch.empty(M, device=dev), torch.empty(M, device=dev)
        self.outputs = [o, n, rs, rp, dy, dr, dwp, dwq, dg]
        self.ws = None
        if own:
            self.ws = torch.empty(swg.residual_norm_bwd_workspace_size(M, N, BF16),
                                  dtype=torch.uint8, device=dev)

    def run(self, stream=None):
        i = self.inputs
        o, n, rs, rp, dy, dr, dwp, dwq, dg = self.outputs
        swg.residual_norm_fwd(i["y"], i["res"], i["wp"], i["w"], i["gate"], 0.5, out=o, norm=n,
                              rstd_post=rs, rstd_pre=rp, stats=True, stream=stream)
        swg.residual_norm_bwd(i["dout"], i["dn"], i["y"], o, i["wp"], i["w"], i["gate"], rs, rp, dy,
                              dr, dwp, dwq, dg, 0.5, workspace=self.ws, stream=stream)


def calls(own):
    """The sizes take every launch: split, packed, whole tiles, few rows, fp32, norms of each form."""
    return {"split": Linear(40, 3000, 264, BF16, "gelu", own=own),
            "packed": Linear(150, 203, 77, FP16, "swish", nk=True, own=own),
            "tiles": Linear(1500, 256, 512, BF16, "none", own=own),
            "few": Linear(4, 520, 264, BF16, "relu", own=own),
            "few nk": Linear(11, 1000, 72, FP32, "gelu_tanh", nk=True, own=own),
            "fp32": Linear(70, 600, 130, FP32, "gelu_tanh", own=own),
            "norm": Norm(500, 768, "channel", own=own), "norm row": Norm(33, 5000, "row", own=own),
            "norm long": Norm(9, 20001, "full", own=own)}


def fill(call, seed):
    """New inputs; returns them, so that they can be put in place later."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    made = {}
    for n, t in call.inputs.items():
        made[n] = torch.randn(t.shape, device="cuda", generator=g)
        made[n] = (made[n] * (call.scale if n == "w" else 1.0)).to(t.dtype)
    return made


def put(call, made):
    for n, t in call.inputs.items():
        t.copy_(made[n])


def eager(call, made):
    put(call, made)
    call.run()
    torch.cuda.synchronize()
    want = [t.clone() for t in call.outputs]
    assert all(t.isfinite().all() for t in want)
    torch.cuda.synchronize()
    return want


def spoil(call):
    for t in (*call.outputs, *call.inputs.values()):
        t.fill_(float("nan"))


@pytest.mark.parametrize("own", [True, False], ids=["own workspace", "allocated"])
def test_streams_that_make_the_inputs(own):
    """The inputs come late on the call's own stream; before, they and the outputs are NaN."""
    runs = calls(own)
    made = {n: fill(c, i) for i, (n, c) in enumerate(runs.items())}
    want = {n: eager(c, made[n]) for n, c in runs.items()}
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    big = torch.randn(2048, 2048, device="cuda")
    for turn in range(2):
        for c in runs.values():
            spoil(c)
        torch.cuda.synchronize()
        for i, (n, c) in enumerate(runs.items()):
            note(f"stream {n}")
            s = side[(i + turn) % 2]
            with torch.cuda.stream(s):
                for _ in range(4):
                    big @ big          # the inputs' producer is behind this
                put(c, made[n])
                if i % 2 == turn:
                    c.run()            # the current stream
            if i % 2 != turn:
                c.run(stream=s)        # a given one
        torch.cuda.synchronize()
        for n, c in runs.items():
            assert all(torch.equal(a, b) for a, b in zip(c.outputs, want[n])), n


@pytest.mark.parametrize("own", [True, False], ids=["own workspace", "allocated"])
def test_graphs_on_new_inputs(own):
    for k, (name, c) in enumerate(calls(own).items()):
        note(f"graph {name}")
        eager(c, fill(c, 100 + k))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            c.run()
        for turn in range(3):
            made = fill(c, 200 + 10 * k + turn)
            want = eager(c, made)
            spoil(c)
            put(c, made)
            torch.randn(500, 500, device="cuda") @ torch.randn(500, 500, device="cuda")
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(c.outputs, want)), (name, turn)


@pytest.mark.parametrize("act", ["none", "gelu"])
def test_outputs_beyond_32_bit_offsets(act):
    """y, z of more than 2^32 bytes: rows at both ends and on either side of 2^31 and 2^32 bytes, none
    like another."""
    M, K, N = (1 << 16) + 133, 16, 1 << 15
    note(f"linear M={M} K={K} N={N} {act}")
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(M, K, device="cuda", generator=g).to(BF16)
    w = (torch.randn(K, N, device="cuda", generator=g) / 4).to(BF16)
    y = torch.full((M, N), float("nan"), dtype=BF16, device="cuda")
    z = torch.full((M, N), float("nan"), dtype=BF16, device="cuda")
    swg.linear_fwd(x, w, act=act, y=y, z=z)
    torch.cuda.synchronize()
    at = 1 << 31 >> 16                      # a row is 2^16 bytes
    for r in (0, at - 140, 2 * at - 140, M - 150):
        rows = slice(r, r + 150)
        ref = x[rows].double() @ w.double()
        # half a step, and sums of 16 products in fp32
        bound = 2.0 ** -8 * ref.abs() + 2.0 ** -20 * (x[rows].double().abs() @ w.double().abs())
        assert ((z[rows].double() - ref).abs() <= bound).all(), r
        if act == "none":
            assert torch.equal(y[rows], z[rows])
        else:
            # the largest slope is 1.13; gelu itself is within 64 roundings of z
            want = torch.nn.functional.gelu(ref)
            bound = 2.0 ** -8 * want.abs() + 1.2 * 2.0 ** -20 * (
                x[rows].double().abs() @ w.double().abs()) + 2.0 ** -18 * ref.abs()
            assert ((y[rows].double() - want).abs() <= bound).all(), r
    assert not y.isnan().any() and not z.isnan().any()
