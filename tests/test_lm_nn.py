"""Shapes that the autograd functions around the linear layers refuse: rows are
flattened before a kernel sees them, so a wrong width must not be regrouped
into other rows."""
import pytest
import torch

from deterministic_invariant_gemm_fwd_gb300 import nn as cnn

D = 8


@pytest.mark.parametrize("x_shape, residual_shape", [
    ((4, 2 * D), None), ((2, 4, D // 2), None), ((), None),
    ((4, D), (2, 2, D)), ((2, 3, D), (3, 2, D)), ((4, D), (1, D)),
])
def test_norm_shapes(x_shape, residual_shape):
    x, gamma, w = torch.zeros(x_shape), torch.ones(D), torch.zeros(D, 16)
    residual = None if residual_shape is None else torch.zeros(residual_shape)
    with pytest.raises(ValueError, match="shape"):
        cnn.rms_norm(x, gamma, residual)
    with pytest.raises(ValueError, match="shape"):
        cnn.norm_linear(x, gamma, w, residual=residual)


@pytest.mark.parametrize("x_shape, targets_shape", [
    ((4, 2 * D), (8,)), ((4, 2 * D), (4,)), ((2, 3, D), (3, 2)), ((2, 3, D), (6,)), ((4, D), (5,)),
])
def test_loss_shapes(x_shape, targets_shape):
    with pytest.raises(ValueError, match="shape"):
        cnn.linear_cross_entropy(torch.zeros(x_shape), torch.zeros(5, D), torch.zeros(targets_shape, dtype=torch.int64))


@pytest.mark.parametrize("padding_idx", [5, -6, 100])
def test_padding_outside(padding_idx):
    with pytest.raises(ValueError, match="padding_idx"):
        cnn.embedding(torch.zeros(3, dtype=torch.int64), torch.zeros(5, D), padding_idx=padding_idx)


@pytest.mark.gpu
@pytest.mark.parametrize("padding_idx, row", [(None, None), (3, 3), (0, 0), (-1, 10), (-11, 0)])
def test_padding_row(padding_idx, row):
    ids = torch.arange(11, device="cuda").repeat(2)
    table = torch.zeros(11, D, device="cuda", requires_grad=True)
    cnn.embedding(ids, table, padding_idx=padding_idx).sum().backward()
    want = torch.full((11, D), 2.0)          # two tokens per row, each adding 1: exact
    if row is not None:
        want[row] = 0
    assert torch.equal(table.grad.cpu(), want)
