"""The b stage refuses column counts whose launch would be cut off."""
from __future__ import annotations

import ctypes

import swish_activation_backward_amd as swg

OK, UNSUPPORTED, WORKSPACE = 0, 3, 4


def test_columns_of_a_launch():
    lib = swg.load_library()
    at = [ctypes.c_void_p((i + 1) << 40) for i in range(8)]

    def call(N, p=at):
        return lib.swiglu_bwd_b(*p[:7], 1, N, 0, p[7], 0, None)

    assert call((1 << 29) + 1) == UNSUPPORTED
    assert call((1 << 29) - 33) == WORKSPACE       # goes on to the next check
    assert call((1 << 29) + 8) == WORKSPACE        # eight at a time
    off = [ctypes.c_void_p(at[0].value + 2), *at[1:]]
    assert call((1 << 29) + 8, off) == UNSUPPORTED
