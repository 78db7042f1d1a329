"""Refusals of the sequence operators' bindings that need no GPU."""
import pytest
import torch

from selective_scan_ss2d_amd import _call, _delta


class Stream:  # stands for one of another GPU
    device = torch.device("cuda", 1)
    cuda_stream = 0


def test_a_stream_of_another_device_is_refused():
    with pytest.raises(ValueError, match="stream is on cuda:1, expected cuda:0"):
        _call.scope(torch.device("cuda", 0), Stream())


@pytest.mark.parametrize("cu", [[0, 4], 4])
def test_offsets_are_a_tensor(cu):
    with pytest.raises(TypeError, match="cu_seqlens"):
        _delta._sequences(cu, 1, torch.device("cuda", 0))
