"""What the binding says to devices that do not fit (no GPU needed)."""
from types import SimpleNamespace

import pytest
import torch

import block_sparse_attention_losa_b200 as losa


def test_a_stream_of_another_device_is_refused():
    """Its kernels would run there, on pointers of the tensors' device."""
    other = SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=0)
    with pytest.raises(ValueError, match="stream"):
        losa._on(other, torch.device("cuda", 0))


def test_host_tensors_are_refused_by_the_layer():
    rope = losa.Rope((2, 3, 4), (16, 24, 24))
    x = torch.zeros(1, 24, 2, 64)
    with pytest.raises(ValueError):
        losa.layer_attn(x, x, x, rope, SimpleNamespace(block=32))


def test_a_pattern_on_the_host_is_refused():
    with pytest.raises(ValueError):
        losa.import_pattern([0, 1], [0], 1, 1, 1, 32, device="cpu")
