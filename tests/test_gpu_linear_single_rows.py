"""The linear layer's C entry points on matrices of a single row, whose stride says nothing."""
from __future__ import annotations

import ctypes

import pytest
import torch

import oracle.ref as R
import swish_activation_backward_amd as swg
from gpu_util import device, note
from linear_models import bwd_models, fwd_models
from parity import to64
from row_models import check

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
TYPES = [BF16, FP16, FP32]


def at(t):
    return ctypes.c_void_p(None if t is None else t.data_ptr())


def workspace(size):
    return torch.empty(max(size, 16), dtype=torch.uint8, device=device())


@pytest.mark.parametrize("ld", ["0", "8", "n + 3"])
@pytest.mark.parametrize("nk", [False, True], ids=["kn", "nk"])
@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("M,K,N", [(1, 64, 72), (1, 4096, 64), (1, 16384, 72), (40, 1, 264),
                                   (40, 264, 1), (1, 1, 1), (1, 520, 1), (1, 1, 520)])
def test_strides_of_single_rows(M, K, N, dt, nk, ld):
    note(f"linear single rows M={M} K={K} N={N} {dt} nk={nk} ld={ld}")
    dev = device()
    g = torch.Generator().manual_seed(M + 3 * K + 5 * N)
    rnd = lambda *s: torch.randn(*s, generator=g).to(dt).to(dev)  # noqa: E731
    x, w, b, res, dy, z = (rnd(M, K), rnd(N, K) if nk else rnd(K, N), rnd(N), rnd(M, N), rnd(M, N),
                           rnd(M, N))
    y, dx, dw, db = (torch.full_like(t, float("nan")) for t in (res, x, w, b))

    def stride(t):   # of the stored rows
        rows, cols = t.shape
        return cols if rows > 1 else {"0": 0, "8": 8, "n + 3": cols + 3}[ld]

    code, act = swg.DTYPE_CODE[dt], swg.ACTIVATION["gelu"]
    lib = swg.load_library()
    stream = torch.cuda.current_stream().cuda_stream
    # the rows there are start at multiples of 16 bytes
    rows16 = all(t.shape[0] == 1 or t.shape[1] * t.element_size() % 16 == 0 for t in (x, w, dy))
    ws = workspace(lib.linear_fwd_workspace_size(M, K, N, nk, code, rows16))
    assert lib.linear_fwd(at(x), stride(x), at(w), stride(w), nk, at(b), at(res), stride(res), at(y),
                          stride(y), None, 0, M, K, N, act, 1.0, code, at(ws), ws.numel(),
                          stream) == 0
    ws = workspace(lib.linear_bwd_workspace_size(M, K, N, nk, act, code, rows16))
    assert lib.linear_bwd(at(dy), stride(dy), at(x), stride(x), at(w), stride(w), nk, at(z),
                          stride(z), at(dx), stride(dx), at(dw), stride(dw), at(db), 0, M, K, N, act,
                          1.0, code, at(ws), ws.numel(), stream) == 0
    torch.cuda.synchronize()
    wkn, dwkn = (w.t(), dw.t()) if nk else (w, dw)
    ry, rz = R.linear_ref(to64(x), to64(wkn), to64(b), to64(res), "gelu", 1.0)
    check("y", y, ry, fwd_models(x, wkn, b, res, "gelu", ry, rz)[0])
    rdx, rdw, rdb, rdz = R.linear_bwd_ref(to64(dy), to64(x), to64(wkn), to64(z), "gelu", 1.0)
    models = bwd_models(dy, x, wkn, z, "gelu", rdz)
    for name, got, ref, e in zip(("dx", "dw", "db"), (dx, dwkn, db), (rdx, rdw, rdb), models):
        check(name, got, ref, e)
