"""What the adapters' module refuses, in words, before a call reaches the
library; no GPU is touched."""
import pytest
import torch

from deterministic_invariant_gemm_fwd_gb300 import nn


def base(K=16, N=24, dtype=torch.bfloat16):
    return nn.Linear(K, N, tier="tc", dtype=dtype)


@pytest.mark.parametrize("rank", [0, -8, 4, 12, 136, 256])
def test_ranks(rank):
    with pytest.raises(ValueError, match="rank"):
        nn.LoraLinear(base(), 2, rank)


@pytest.mark.parametrize("rank", [8, 24, 128])
def test_ranks_that_are_taken(rank):
    layer = nn.LoraLinear(base(), 2, rank)
    assert layer.a.shape == (2, 16, rank) and layer.b.shape == (2, rank, 24)


def test_numbers_of_adapters():
    with pytest.raises(ValueError, match="adapters"):
        nn.LoraLinear(base(), 0, 8)


@pytest.mark.parametrize("K,N", [(12, 24), (16, 20)])
def test_widths(K, N):
    with pytest.raises(ValueError, match="multiples of 8"):
        nn.LoraLinear(base(K, N), 2, 8)


def test_float32_layers():
    layer = nn.LoraLinear(base(dtype=torch.float32), 2, 8)       # may be cast before it is called
    with pytest.raises(TypeError, match="bfloat16 or float16"):
        layer(torch.zeros(4, 16), torch.zeros(4, dtype=torch.int64))
    with pytest.raises(TypeError, match="bfloat16 or float16"):
        layer(torch.zeros(4, 16), 1)


@pytest.mark.parametrize("adapter", [2, -2, 10 ** 12])
def test_a_number_that_names_no_adapter(adapter):
    layer = nn.LoraLinear(base(), 2, 8)
    with pytest.raises(ValueError, match="adapter"):
        layer(torch.zeros(4, 16, dtype=torch.bfloat16), adapter)
