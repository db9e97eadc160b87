"""The norm that clip_grad_norm_ returns where no parameter has a gradient."""
import torch

from deterministic_invariant_gemm_fwd_gb300 import nn


def test_the_norm_is_on_the_parameters_device():
    meta = [torch.nn.Parameter(torch.zeros(3, device="meta")), torch.nn.Parameter(torch.zeros(2, device="meta"))]
    for parameters in (meta, iter(meta), meta[0]):
        norm = nn.clip_grad_norm_(parameters, 1.0)
        assert norm.device.type == "meta" and norm.shape == () and norm.dtype is torch.float32
    assert float(nn.clip_grad_norm_([], 1.0)) == 0.0
