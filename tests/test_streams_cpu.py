"""A stream of another device than the tensors' is refused.  Without a GPU: the tensors have a
device and no storage, the streams are stand-ins."""
from __future__ import annotations

from types import SimpleNamespace

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import swish_activation_backward_amd as swg
from swish_activation_backward_amd import _lib

DEVICE, OTHER = torch.device("cuda", 0), torch.device("cuda", 1)


@pytest.mark.parametrize("call", [
    lambda x, f, ids, s: swg.layer_norm_fwd(x, None, None, stream=s),
    lambda x, f, ids, s: swg.layer_norm_bwd(x, x, None, f, f, None, f, f, stream=s),
    lambda x, f, ids, s: swg.token_logprobs(x, stream=s),
    lambda x, f, ids, s: swg.token_logprobs_bwd(x, None, f, f, None, f, stream=s),
    lambda x, f, ids, s: swg.distill_fwd(x, x, ids, stream=s),
    lambda x, f, ids, s: swg.distill_bwd(x, x, ids, f, f, stream=s),
    lambda x, f, ids, s: swg.distill_fwd_bwd(x, x, ids, f, stream=s),
], ids=["layer_norm_fwd", "layer_norm_bwd", "token_logprobs", "token_logprobs_bwd", "distill_fwd",
        "distill_bwd", "distill_fwd_bwd"])
def test_row_operators_refuse_a_stream_of_another_device(call):
    with FakeTensorMode():
        x = torch.empty(4, 8, device=DEVICE)
        f = torch.empty(4, device=DEVICE)
        ids = torch.empty(4, 8, dtype=torch.int64, device=DEVICE)
    with pytest.raises(ValueError, match="stream of cuda:1"):
        call(x, f, ids, SimpleNamespace(device=OTHER, cuda_stream=1))


def test_stream_handles_are_of_the_tensors_device():
    assert _lib._stream(SimpleNamespace(device=DEVICE, cuda_stream=7), DEVICE) == 7
    with pytest.raises(ValueError, match="stream of cuda:1"):
        _lib._stream(SimpleNamespace(device=OTHER, cuda_stream=7), DEVICE)


def test_host_tensors_are_named_before_the_stream():
    with pytest.raises(ValueError, match="GPU only"):
        swg.token_logprobs(torch.zeros(2, 3), stream=SimpleNamespace(device=DEVICE, cuda_stream=1))
