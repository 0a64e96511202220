"""The autograd wrappers' view of their operands as matrices."""
from __future__ import annotations

import pytest
import torch

from swish_activation_backward_amd.autograd import _rows_of


@pytest.mark.parametrize("shape,want", [((5,), (1, 5)), ((2, 3, 5), (6, 5)), ((2, 3, 0), (6, 0)),
                                        ((0, 3, 5), (0, 5)), ((2, 0, 0), (0, 0)), ((0,), (1, 0)),
                                        ((4, 1), (4, 1))])
def test_shapes(shape, want):
    assert _rows_of(torch.empty(shape)).shape == want


def test_rows_are_taken_where_they_lie():
    x = torch.arange(60.0).view(6, 10)
    assert _rows_of(x[:, :7]).data_ptr() == x.data_ptr()
    for t in (x.t(), x[:, ::2], x[:1].expand(6, 10)):
        r = _rows_of(t)
        assert torch.equal(r, t) and r.is_contiguous()
