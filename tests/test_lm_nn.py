"""Shapes that the autograd functions around the linear layers refuse: rows are
flattened before a kernel sees them, so a wrong width must not be regrouped
into other rows."""
import pytest
import torch

import deterministic_invariant_gemm_fwd_gb300 as cg
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


# ---- the autograd functions with plain CPU stand-ins for the kernels ---------------

def _fwd(x, gamma, residual=None, eps=1e-6, quantize=False):
    h = x if residual is None else x + residual
    rstd = (h.square().mean(1) + eps).rsqrt()
    n = h * rstd[:, None]
    return cg.RmsNorm(n * gamma, h, rstd, n if quantize else None, torch.ones_like(rstd) if quantize else None)


def _bwd(dy, gamma, rstd, h=None, codes=None, scales=None, dh=None, recompute=False):
    n = codes if h is None else h * rstd[:, None]
    dx = rstd[:, None] * (gamma * dy - n * (gamma * dy * n).mean(1, keepdim=True)) + (0 if dh is None else dh)
    return (dx, (dy * n).sum(0)) + ((n * gamma,) if recompute else ())


@pytest.fixture
def stand_ins(monkeypatch):
    calls = []

    def bwd(*args, **kw):
        calls.append(kw)
        return _bwd(*args, **kw)

    monkeypatch.setattr(cnn, "rms_norm_fwd", _fwd)
    monkeypatch.setattr(cnn, "rms_norm_bwd", bwd)
    monkeypatch.setattr(cnn, "linear_fwd", lambda x, w, b, tier: x @ w + (0 if b is None else b))
    monkeypatch.setattr(cnn, "linear_dx", lambda g, w, tier: g @ w.t())
    monkeypatch.setattr(cnn, "linear_dw", lambda x, g, tier: x.t() @ g)
    monkeypatch.setattr(cnn, "bias_grad", lambda g, tier: g.sum(0))
    monkeypatch.setattr(cnn, "embedding_fwd", lambda table, ids, scale: scale * table[ids])
    monkeypatch.setattr(cnn, "embedding_bwd", lambda dy, ids, rows, scale, pad: scale * torch.zeros(
        rows, dy.shape[-1]).index_add_(0, ids.reshape(-1), dy.reshape(-1, dy.shape[-1])))
    monkeypatch.setattr(cnn, "linear_cross_entropy_fwd", lambda x, w, t, i, r: (
        torch.nn.functional.cross_entropy(x @ w.t(), t, ignore_index=i, reduction=r), torch.logsumexp(x @ w.t(), 1)))
    monkeypatch.setattr(cnn, "linear_cross_entropy_bwd", lambda g, x, w, t, lse, i, r: (
        torch.zeros_like(x) + g.sum(), torch.zeros_like(w) + g.sum()))
    return calls


def _leaves(*shapes):
    g = torch.Generator().manual_seed(1)
    return [torch.randn(s, generator=g).requires_grad_() for s in shapes]


def test_gradients_of_gradients_raise(stand_ins):
    """Also where the incoming gradient is a constant, as a loss's is."""
    x, res, gamma, w, b, table = _leaves((4, D), (4, D), (D,), (D, 3), (3,), (5, D))
    ids = torch.tensor([0, 4, 4, 1])
    cases = [(lambda: cnn.embedding(ids, table), [table]), (lambda: cnn.rms_norm(x, gamma), [x, gamma]),
             (lambda: cnn.rms_norm(x, gamma, res)[0], [x, res, gamma]),
             (lambda: cnn.norm_linear(x, gamma, w, b), [x, gamma, w, b]),
             (lambda: cnn.linear_cross_entropy(x, table, ids), [x, table])]
    for make, leaves in cases:
        for power in (1, 2):
            for k in range(len(leaves)):
                out = make().pow(power).sum()
                g = torch.autograd.grad(out, leaves, create_graph=True)
                plain = torch.autograd.grad(make().pow(power).sum(), leaves)
                assert all(torch.equal(a, p) for a, p in zip(g, plain))
                with pytest.raises(RuntimeError, match="no derivative"):
                    (out + g[k].square().sum()).backward()


@pytest.mark.parametrize("layer", ["norm", "norm_linear"])
def test_outputs_that_go_nowhere(stand_ins, layer):
    """The last norm's residual stream has no gradient: none is made up and
    read.  Nor does a norm of which only the residual stream goes on run its
    gradient; what it would have given is zero."""
    shapes = [(2, 3, D), (2, 3, D), (D,)] + ([(D, 4), (4,)] if layer == "norm_linear" else [])

    def grads(used, other):
        leaves = _leaves(*shapes)
        x, res, gamma, *rest = leaves
        outs = cnn.norm_linear(x, gamma, *rest, residual=res) if rest else cnn.rms_norm(x, gamma, res)
        total = outs[used].sum()
        (total + other * outs[1 - used].sum() if other is not None else total).backward()
        return [leaf.grad for leaf in leaves]

    for used in (0, 1):
        stand_ins.clear()
        alone = grads(used, None)
        assert [c["dh"] for c in stand_ins] == ([None] if used == 0 else [])
        stand_ins.clear()
        both = grads(used, 0.0)
        assert len(stand_ins) == 1 and stand_ins[0]["dh"] is not None
        assert all(a.shape == b.shape and torch.equal(a, b) for a, b in zip(alone, both))
