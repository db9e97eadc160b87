"""What the modules leave out: the adapters' u where no gradient is wanted."""
import pytest
import torch

from deterministic_invariant_gemm_fwd_gb300 import nn


@pytest.fixture
def kept(monkeypatch):
    """The `keep` of every forward call; y is zeros."""
    calls = []

    def fwd(x, weight, a, b, adapters, scales, bias=None, keep=False, stream=None):
        calls.append(keep)
        y = torch.zeros(x.shape[0], weight.shape[1], dtype=x.dtype)
        return (y, torch.zeros(x.shape[0], 3, 16, dtype=x.dtype)) if keep else y
    monkeypatch.setattr(nn, "lora_linear_fwd", fwd)
    return calls


def test_u_is_kept_for_a_gradient_alone(kept):
    layer = nn.LoraLinear(nn.Linear(16, 24, tier="tc", dtype=torch.bfloat16), 2, 8)
    x, ids = torch.zeros(2, 5, 16, dtype=torch.bfloat16), torch.zeros(2, 5, dtype=torch.int64)
    y = layer(x, ids)
    assert kept == [True] and y.requires_grad and y.shape == (2, 5, 24)
    with torch.no_grad():
        y = layer(x, ids)
    assert kept == [True, False] and not y.requires_grad and y.shape == (2, 5, 24)
    for p in layer.parameters():
        p.requires_grad_(False)
    y = layer(x, ids)
    assert kept == [True, False, False] and not y.requires_grad
    y = layer(x.clone().requires_grad_(), ids)
    assert kept[3:] == [True] and y.requires_grad
