"""The temperatures that the operators on logits take, without a GPU (no call reaches a launch)."""
from __future__ import annotations

import pytest

from test_rows_cpu import (INVALID, OK, distill_both, distill_bwd, distill_fwd, lib,  # noqa: F401
                           logprobs, logprobs_bwd)


@pytest.mark.parametrize("call", [logprobs, logprobs_bwd, distill_fwd, distill_bwd, distill_both])
def test_scale_of_the_temperature_is_finite(lib, call):   # noqa: F811
    """1 / 3e-39 is a finite fp32 number, log2(e) / 3e-39 is not: a row's largest logit would
    meet it as 0 times infinity."""
    for t in (3e-39, 4e-39, 4.2e-39):
        assert call(lib, t=t) == INVALID, t
        assert call(lib, t=t, R=0) == INVALID, t
    for t in (4.3e-39, 1e-38, 1e38):
        assert call(lib, t=t, R=0) == OK, t
