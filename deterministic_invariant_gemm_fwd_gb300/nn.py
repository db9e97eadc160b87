"""Autograd linear layer over the carbon_gemm C ABI.

A drop-in linear layer whose three GEMMs run in this library's kernels, as
the sgemm-bi page describes its ``Linear`` module and functional form
("Use": weights stored [in, out], ``Linear.from_torch`` converting a
``torch.nn.Linear``; the tensor-core switch there is the ``tier`` argument
here) and as the Carbon README describes its ``DeterministicLinear`` ("How
It Works").

    forward   Y  = X.W + b       carbon_gemm_fwd
    backward  dX = dY.W^T        carbon_gemm_dx
              dW = X^T.dY        carbon_gemm_dw
              db = sum_t dY[t]   carbon_gemm_dw with a column of ones for X,
                                 on the exact tier (on the correctly
                                 rounded tier when the layer uses it)

The bias gradient is the one piece the sgemm-bi page leaves to a plain
PyTorch column sum ("Determinism contracts"); here it is the exact tier's
fixed-order sum over tokens (256-token chunks summed with KBN, the chunk
values combined with KBN, one rounding), so it is bit-identical run to run,
for every batch split into the same tokens, and to the CPU oracle.  A layer
on the correctly rounded tier ("superacc") takes db from that tier too: the
exact column sum rounded once.

Around the linear layers: ``Embedding`` / ``embedding``, ``RMSNorm`` /
``rms_norm``, ``norm_linear`` (norm and linear layer with an 8-bit
checkpoint) and ``linear_cross_entropy`` (output layer and loss), each with a
deterministic gradient.

Leading dimensions of the input are flattened into the token dimension.
There is no CPU path: inputs must be CUDA tensors (float32, bfloat16 or
float16; the tensor-core tier takes bfloat16 or float16).
"""
from __future__ import annotations

import functools
import math

import torch

from . import (_dtype_code, carbon_gemm_dw, embedding_bwd, embedding_fwd,
               linear_cross_entropy_bwd, linear_cross_entropy_fwd, linear_dw, linear_dx, linear_fwd,
               rms_norm_bwd, rms_norm_fwd)


def bias_grad(dY, stream=None, tier="exact"):
    """db[N] = sum over tokens t of dY[t, :]: the GEMM dW = X^T.dY with X a
    column of ones (every product is exact), in dY's dtype, on the exact tier
    (fixed-order KBN) or, with tier="superacc", correctly rounded."""
    if tier not in ("exact", "superacc"):
        raise ValueError("the bias gradient runs on the exact or the superacc tier")
    if dY.dim() != 2 or not dY.is_contiguous() or not dY.is_cuda:
        raise ValueError("dY must be a contiguous 2-D CUDA tensor")
    M, N = dY.shape
    ones = torch.ones((M, 1), dtype=dY.dtype, device=dY.device)
    db = torch.empty((1, N), dtype=dY.dtype, device=dY.device)
    carbon_gemm_dw(db, ones, dY, M, 1, N, _dtype_code(dY), tier, stream)
    return db.view(N)


class _LinearFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, tier):
        K, N = weight.shape
        if x.shape[-1] != K:
            raise ValueError(f"input has {x.shape[-1]} features, weight expects {K}")
        x2 = x.reshape(-1, K).contiguous()
        y = linear_fwd(x2, weight, bias, tier)
        ctx.save_for_backward(x2, weight)
        ctx.tier = tier
        ctx.has_bias = bias is not None
        ctx.x_shape = x.shape
        return y.view(*x.shape[:-1], N)

    @staticmethod
    def backward(ctx, grad_y):
        x2, weight = ctx.saved_tensors
        g2 = grad_y.reshape(-1, weight.shape[1]).contiguous()
        dx = dw = db = None
        if ctx.needs_input_grad[0]:
            dx = linear_dx(g2, weight, ctx.tier).view(ctx.x_shape)
        if ctx.needs_input_grad[1]:
            dw = linear_dw(x2, g2, ctx.tier)
        if ctx.has_bias and ctx.needs_input_grad[2]:
            db = bias_grad(g2, tier="superacc" if ctx.tier == "superacc" else "exact")
        return dx, dw, db, None


def deterministic_linear(x, weight, bias=None, tier="exact"):
    """y = x.weight + bias with weight [in, out]; differentiable in x, weight
    and bias (the gradients come from the same library)."""
    return _LinearFunction.apply(x, weight, bias, tier)


class Linear(torch.nn.Module):
    """Linear layer with weight [in_features, out_features] and the library's
    kernels for the forward and backward GEMMs."""

    def __init__(self, in_features, out_features, bias=True, tier="exact", device=None,
                 dtype=None):
        super().__init__()
        self.in_features, self.out_features, self.tier = in_features, out_features, tier
        self.weight = torch.nn.Parameter(torch.empty((in_features, out_features), device=device,
                                                     dtype=dtype))
        self.bias = (torch.nn.Parameter(torch.empty(out_features, device=device, dtype=dtype))
                     if bias else None)
        self.reset_parameters()

    def reset_parameters(self):
        # torch.nn.Linear's initialisation, applied to the [out, in] view
        torch.nn.init.kaiming_uniform_(self.weight.t(), a=math.sqrt(5))
        if self.bias is not None:
            bound = 1.0 / math.sqrt(self.in_features) if self.in_features > 0 else 0.0
            torch.nn.init.uniform_(self.bias, -bound, bound)

    @classmethod
    def from_torch(cls, linear: torch.nn.Linear, tier="exact"):
        """The same layer with its weight stored [in, out] (a copy)."""
        out = cls(linear.in_features, linear.out_features, bias=linear.bias is not None,
                  tier=tier, device=linear.weight.device, dtype=linear.weight.dtype)
        with torch.no_grad():
            out.weight.copy_(linear.weight.t())
            if linear.bias is not None:
                out.bias.copy_(linear.bias)
        return out

    def forward(self, x):
        return deterministic_linear(x, self.weight, self.bias, self.tier)

    def extra_repr(self):
        return (f"in_features={self.in_features}, out_features={self.out_features}, "
                f"bias={self.bias is not None}, tier={self.tier!r}")


# ---- the operators around the linear layers -------------------------------------


class _NoDerivative(torch.autograd.Function):
    """Its first n tensors, from all of them; differentiating raises."""

    @staticmethod
    def forward(ctx, n, *tensors):
        return tuple(t.view_as(t) for t in tensors[:n])

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError("the gradients of this package's operators have no derivative of their own")


def _once(backward):
    """A backward pass that can be differentiated once: with create_graph=True
    its results raise where a second derivative reaches them (as constants,
    which is what kernels return, they would drop out of it unseen)."""
    @functools.wraps(backward)
    def run(ctx, *grads):
        with torch.no_grad():
            out = backward(ctx, *grads)
        if not torch.is_grad_enabled():
            return out
        behind = [t for t in (*ctx.saved_tensors, *grads) if t is not None and t.requires_grad]
        made = [t.detach().requires_grad_() for t in out if t is not None]
        made = iter(_NoDerivative.apply(len(made), *made, *behind))
        return tuple(None if t is None else next(made) for t in out)
    return run


class _EmbeddingFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ids, table, scale, padding_idx):
        ctx.save_for_backward(ids)
        ctx.rows, ctx.scale, ctx.padding_idx = table.shape[0], scale, padding_idx
        return embedding_fwd(table, ids, scale)

    @staticmethod
    @_once
    def backward(ctx, grad):
        (ids,) = ctx.saved_tensors
        return None, embedding_bwd(grad.contiguous(), ids, ctx.rows, ctx.scale, ctx.padding_idx), None, None


def embedding(ids, table, scale=1.0, padding_idx=None):
    """scale * table[ids], differentiable in table; the gradient adds a row's
    tokens in the order of their positions (no atomics).  The row padding_idx
    (negative: counted from the end) gets no gradient."""
    padding = -1
    if padding_idx is not None:
        rows = table.shape[0]
        if not -rows <= padding_idx < rows:
            raise ValueError(f"padding_idx {padding_idx} is outside a table of {rows} rows")
        padding = padding_idx % rows
    return _EmbeddingFunction.apply(ids.contiguous(), table, float(scale), padding)


class Embedding(torch.nn.Module):
    """Token embedding [num_rows, width] with an output scale.  Its weight can
    be the table of linear_cross_entropy as well (tied weights)."""

    def __init__(self, num_rows, width, scale=1.0, padding_idx=None, device=None, dtype=None):
        super().__init__()
        self.scale, self.padding_idx = scale, padding_idx
        self.weight = torch.nn.Parameter(torch.empty((num_rows, width), device=device, dtype=dtype))
        torch.nn.init.normal_(self.weight, std=0.02)

    def forward(self, ids):
        return embedding(ids, self.weight, self.scale, self.padding_idx)

    def extra_repr(self):
        return f"{self.weight.shape[0]}, {self.weight.shape[1]}, scale={self.scale}, padding_idx={self.padding_idx}"


def _flat(t, width):
    return t.reshape(-1, width).contiguous()


def _width(x, width, residual=None):
    """Raises unless x has rows of this width, and residual x's shape: rows
    are flattened, which would regroup the elements of others."""
    if x.dim() < 1 or x.shape[-1] != width:
        raise ValueError(f"x has shape {tuple(x.shape)}; expected [..., {width}]")
    if residual is not None and residual.shape != x.shape:
        raise ValueError(f"residual has shape {tuple(residual.shape)}, x {tuple(x.shape)}")


class _RmsNormFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, gamma, eps):
        D = gamma.shape[0]
        r = rms_norm_fwd(_flat(x, D), gamma, None if residual is None else _flat(residual, D), eps)
        ctx.save_for_backward(r.h, r.rstd, gamma)
        ctx.shape, ctx.has_residual = x.shape, residual is not None
        ctx.set_materialize_grads(False)        # an output that goes nowhere: None, not a tensor of zeros
        y = r.y.view(x.shape)
        return (y, r.h.view(x.shape)) if ctx.has_residual else y

    @staticmethod
    @_once
    def backward(ctx, dy, dh=None):
        h, rstd, gamma = ctx.saved_tensors
        D = gamma.shape[0]
        if dy is None:                          # only the residual stream goes on
            return dh, dh if ctx.has_residual else None, torch.zeros_like(gamma), None
        dx, dgamma = rms_norm_bwd(_flat(dy, D), gamma, rstd, h=h, dh=None if dh is None else _flat(dh, D))
        dx = dx.view(ctx.shape)
        return dx, dx if ctx.has_residual else None, dgamma, None


def rms_norm(x, gamma, residual=None, eps=1e-6):
    """y = norm(x + residual) * gamma over the last dimension; with a residual
    returns (y, x + residual), the second being the residual stream that goes
    on.  Differentiable in x, residual and gamma."""
    _width(x, gamma.shape[0], residual)
    return _RmsNormFunction.apply(x, residual, gamma, eps)


class RMSNorm(torch.nn.Module):
    """Root-mean-square norm over the last dimension; forward(x) -> y,
    forward(x, residual) -> (y, x + residual)."""

    def __init__(self, width, eps=1e-6, device=None, dtype=None):
        super().__init__()
        self.eps = eps
        self.weight = torch.nn.Parameter(torch.ones(width, device=device, dtype=dtype))

    def forward(self, x, residual=None):
        return rms_norm(x, self.weight, residual, self.eps)

    def extra_repr(self):
        return f"{self.weight.shape[0]}, eps={self.eps}"


class _NormLinearFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, gamma, weight, bias, eps, tier):
        D = gamma.shape[0]
        r = rms_norm_fwd(_flat(x, D), gamma, None if residual is None else _flat(residual, D), eps, quantize=True)
        out = linear_fwd(r.y, weight, bias, tier)
        ctx.save_for_backward(r.codes, r.scales, r.rstd, gamma, weight)
        ctx.shape, ctx.tier, ctx.has_bias, ctx.has_residual = x.shape, tier, bias is not None, residual is not None
        ctx.set_materialize_grads(False)
        out = out.view(*x.shape[:-1], weight.shape[1])
        return (out, r.h.view(x.shape)) if ctx.has_residual else out

    @staticmethod
    @_once
    def backward(ctx, dout, dh=None):
        codes, scales, rstd, gamma, weight = ctx.saved_tensors
        D = gamma.shape[0]
        if dout is None:
            db = weight.new_zeros(weight.shape[1]) if ctx.has_bias else None
            return dh, dh if ctx.has_residual else None, torch.zeros_like(gamma), torch.zeros_like(weight), db, None, None
        g = _flat(dout, weight.shape[1])
        dy = linear_dx(g, weight, ctx.tier)
        dx, dgamma, y = rms_norm_bwd(dy, gamma, rstd, codes=codes, scales=scales,
                                     dh=None if dh is None else _flat(dh, D), recompute=True)
        dw = linear_dw(y, g, ctx.tier) if ctx.needs_input_grad[3] else None
        db = None
        if ctx.has_bias and ctx.needs_input_grad[4]:
            db = bias_grad(g, tier="superacc" if ctx.tier == "superacc" else "exact")
        dx = dx.view(ctx.shape)
        return dx, dx if ctx.has_residual else None, dgamma, dw, db, None, None


def norm_linear(x, gamma, weight, bias=None, residual=None, eps=1e-6, tier="exact"):
    """deterministic_linear(rms_norm(x + residual), weight, bias) that keeps,
    for the backward pass, the normalised rows in 8 bits with a scale per
    token instead of the residual stream and the linear layer's input: one
    byte per element where rms_norm followed by deterministic_linear keeps
    two tensors of the input's type.  The forward pass is the same; the
    backward pass reads the rows back to within scale / 2 = max|row| / 254.
    With a residual returns (output, x + residual)."""
    _width(x, gamma.shape[0], residual)
    return _NormLinearFunction.apply(x, residual, gamma, weight, bias, eps, tier)


class _LinearCrossEntropyFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, table, targets, ignore_index, reduction):
        x2 = _flat(x, table.shape[1])
        t = targets.reshape(-1).contiguous()
        loss, lse = linear_cross_entropy_fwd(x2, table, t, ignore_index, reduction)
        ctx.save_for_backward(x2, table, t, lse)
        ctx.shape, ctx.ignore_index, ctx.reduction = x.shape, ignore_index, reduction
        return loss.view(targets.shape) if reduction == "none" else loss

    @staticmethod
    @_once
    def backward(ctx, grad):
        x2, table, t, lse = ctx.saved_tensors
        g = grad.reshape(-1).contiguous() if ctx.reduction == "none" else grad
        dx, dtable = linear_cross_entropy_bwd(g, x2, table, t, lse, ctx.ignore_index, ctx.reduction)
        return dx.view(ctx.shape), dtable, None, None, None


def linear_cross_entropy(x, table, targets, ignore_index=-100, reduction="mean"):
    """Softmax cross entropy of the logits x . table^T (table [V, D], e.g. an
    Embedding's weight) against targets, without storing the logits;
    differentiable in x and table.  reduction="mean" divides by the positions
    that count and is 0 where there are none."""
    _width(x, table.shape[1])
    if targets.shape != x.shape[:-1]:
        raise ValueError(f"targets has shape {tuple(targets.shape)}; expected {tuple(x.shape[:-1])}")
    return _LinearCrossEntropyFunction.apply(x, table, targets, ignore_index, reduction)
