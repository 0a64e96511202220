"""The linear layer's checks without a GPU where a matrix has a single row."""
from __future__ import annotations

import pytest

import swish_activation_backward_amd as swg
from test_linear_cpu import BF16, INVALID, WORKSPACE, addr, bwd, fwd


@pytest.fixture(scope="module")
def lib():
    return swg.load_library()


def test_a_single_rows_stride_takes_no_workspace(lib):
    """A single row at a multiple of 16 bytes needs what the query says, whatever its stride is.  (An
    output over an input is refused behind the workspace's size, so that nothing is launched.)"""
    for M, K, N, nk, ld in ((1, 4096, 64, 0, dict(ldx=4099)), (40, 1, 264, 0, dict(ldw=267)),
                            (40, 264, 1, 1, dict(ldw=267))):
        size = lib.linear_fwd_workspace_size(M, K, N, nk, BF16, 1)
        a = dict(M=M, K=K, N=N, nk=nk, ldx=K, ldw=K if nk else N, ldr=N, ldy=N, ldz=N, wsb=size,
                 y=addr(0))
        a.update(ld)
        assert fwd(lib, **a) == INVALID, ld
        assert size == 0 or fwd(lib, **{**a, "wsb": size - 1}) == WORKSPACE
    size = lib.linear_bwd_workspace_size(1, 4096, 64, 0, 0, BF16, 1)
    a = dict(M=1, K=4096, N=64, act=0, ldx=4099, ldw=64, lddy=67, lddx=4096, lddw=64, wsb=size)
    assert bwd(lib, **a, dx=addr(0)) == INVALID
    assert size > 0 and bwd(lib, **{**a, "wsb": size - 1}, dx=addr(0)) == WORKSPACE
