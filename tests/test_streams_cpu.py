"""The checks of the stream argument that need no GPU."""
import types

import pytest
import torch

import mixture_experts_ffn_10_b200 as moe


def test_a_stream_of_another_device_is_refused():
    stream = types.SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=0)
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        moe._on(torch.device("cuda", 0), stream)


def test_tensors_off_the_gpu_are_refused():
    for stream in (None, types.SimpleNamespace(device=torch.device("cuda", 0), cuda_stream=0)):
        with pytest.raises(ValueError, match="CUDA device"):
            moe._on(torch.device("cpu"), stream)
