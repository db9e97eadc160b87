"""The operators around a language model's linear layers as functions of
torch tensors (``include/carbon_lm.h``): token embedding, root-mean-square
norm with an 8-bit checkpoint, and the output layer's softmax cross entropy.

Each function checks its arguments, allocates the outputs and the workspace
with torch's allocator and makes the library call on ``stream`` (default:
the current stream).  Nothing is copied or converted: operands are contiguous
CUDA tensors on the current device, token ids and targets int64.  ``nn`` wraps
the functions in autograd.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

from . import _binding as _b


_CODES = {"torch.float32": _b.F32, "torch.bfloat16": _b.BF16, "torch.float16": _b.F16}


def _dtype(name, t):
    code = _CODES.get(str(t.dtype))
    if code is None:
        raise TypeError(f"{name} has dtype {t.dtype}; expected float32, bfloat16 or float16")
    return code


def _need(name, t, shape, dtype):
    """A contiguous CUDA tensor of this shape and dtype."""
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")


def _rows(name, t):
    if t.dim() != 2 or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous 2-D CUDA tensor")
    return t.shape


class _Launch:
    """The stream of a call: its handle, and the outputs and workspace that
    belong to it.  On a stream other than the current one the workspace is
    taken under that stream, and the outputs are marked as used there, so
    that the allocator hands neither out again while the kernels run."""

    def __init__(self, stream):
        import torch
        current = torch.cuda.current_stream()
        if stream is None:
            stream = current
        elif isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
        self.stream, self.handle = stream, stream.cuda_stream
        self.other = self.handle != current.cuda_stream

    def out(self, shape, dtype, device):
        import torch
        t = torch.empty(shape, dtype=dtype, device=device)
        if self.other:
            t.record_stream(self.stream)
        return t

    def workspace(self, nbytes, device):
        import torch
        if nbytes < 0:
            raise ValueError("sizes out of range")
        if not self.other:
            return torch.empty(max(nbytes, 16), dtype=torch.uint8, device=device)
        with torch.cuda.stream(self.stream):
            return torch.empty(max(nbytes, 16), dtype=torch.uint8, device=device)


def embedding_fwd(table, ids, scale=1.0, stream=None):
    """scale * table[ids]: table [V, D], ids int64 of any shape -> [*ids.shape, D]."""
    import torch
    V, D = _rows("table", table)
    _need("ids", ids, ids.shape, torch.int64)
    L = _Launch(stream)
    out = L.out((*ids.shape, D), table.dtype, table.device)
    _b.carbon_embedding_fwd(out, table, ids, ids.numel(), V, D, scale, _dtype("table", table), L.handle)
    return out


def embedding_bwd(dy, ids, num_rows, scale=1.0, padding_idx=-1, accumulate_to=None, stream=None):
    """Gradient of the table: [num_rows, D] from dy [*ids.shape, D].  With
    accumulate_to (a gradient of the same table, e.g. the output layer's) the
    sums are added to it in place and it is returned."""
    import torch
    D = dy.shape[-1]
    _need("ids", ids, ids.shape, torch.int64)
    _need("dy", dy, (*ids.shape, D), dy.dtype)
    code = _dtype("dy", dy)
    L = _Launch(stream)
    if accumulate_to is None:
        out = L.out((num_rows, D), dy.dtype, dy.device)
    else:
        out = accumulate_to
        _need("accumulate_to", out, (num_rows, D), dy.dtype)
    M = ids.numel()
    nbytes = _b.carbon_embedding_bwd_workspace(M, num_rows, D)
    ws = L.workspace(nbytes, dy.device)
    _b.carbon_embedding_bwd(out, dy, ids, M, num_rows, D, scale, padding_idx, accumulate_to is not None,
                            ws, nbytes, code, L.handle)
    return out


class RmsNorm(NamedTuple):
    """What rms_norm_fwd returns; codes and scales are None without quantize."""
    y: object                    # norm(x + residual) * gamma
    h: object                    # x + residual (x itself without a residual)
    rstd: object                 # fp32 [M]
    codes: Optional[object]      # int8 [M, D]
    scales: Optional[object]     # fp32 [M]


def rms_norm_fwd(x, gamma, residual=None, eps=1e-6, quantize=False, stream=None):
    """RMS norm of x + residual, [M, D]; quantize=True also writes the 8-bit
    checkpoint of the normalised rows."""
    import torch
    M, D = _rows("x", x)
    code = _dtype("x", x)
    _need("gamma", gamma, (D,), x.dtype)
    L = _Launch(stream)
    h = x
    if residual is not None:
        _need("residual", residual, (M, D), x.dtype)
        h = L.out((M, D), x.dtype, x.device)
    y = L.out((M, D), x.dtype, x.device)
    rstd = L.out((M,), torch.float32, x.device)
    codes = scales = None
    if quantize:
        codes = L.out((M, D), torch.int8, x.device)
        scales = L.out((M,), torch.float32, x.device)
    _b.carbon_rms_norm_fwd(y, None if residual is None else h, rstd, codes, scales, x, residual, gamma, M, D,
                           eps, code, L.handle)
    return RmsNorm(y, h, rstd, codes, scales)


def rms_norm_bwd(dy, gamma, rstd, h=None, codes=None, scales=None, dh=None, recompute=False, stream=None):
    """(dx, dgamma) of rms_norm_fwd from h, or from codes and scales; dx is
    the gradient of x and of the residual.  dh: the gradient that reaches h
    from further on.  recompute=True returns (dx, dgamma, y)."""
    import torch
    M, D = _rows("dy", dy)
    code = _dtype("dy", dy)
    _need("gamma", gamma, (D,), dy.dtype)
    _need("rstd", rstd, (M,), torch.float32)
    if (h is None) == (codes is None) or (codes is None) != (scales is None):
        raise ValueError("give either h, or codes and scales")
    if h is not None:
        _need("h", h, (M, D), dy.dtype)
    else:
        _need("codes", codes, (M, D), torch.int8)
        _need("scales", scales, (M,), torch.float32)
    if dh is not None:
        _need("dh", dh, (M, D), dy.dtype)
    L = _Launch(stream)
    dx = L.out((M, D), dy.dtype, dy.device)
    dgamma = L.out((D,), dy.dtype, dy.device)
    y = L.out((M, D), dy.dtype, dy.device) if recompute else None
    nbytes = _b.carbon_rms_norm_bwd_workspace(M, D)
    ws = L.workspace(nbytes, dy.device)
    _b.carbon_rms_norm_bwd(dx, dgamma, y, dy, h, codes, scales, rstd, gamma, dh, M, D, ws, nbytes, code, L.handle)
    return (dx, dgamma, y) if recompute else (dx, dgamma)


def rms_norm_expand(codes, scales, gamma=None, dtype=None, stream=None):
    """codes * scales (* gamma) in dtype (gamma's, or bfloat16)."""
    import torch
    M, D = _rows("codes", codes)
    _need("codes", codes, (M, D), torch.int8)
    _need("scales", scales, (M,), torch.float32)
    dtype = dtype or (gamma.dtype if gamma is not None else torch.bfloat16)
    if gamma is not None:
        _need("gamma", gamma, (D,), dtype)
    L = _Launch(stream)
    out = L.out((M, D), dtype, codes.device)
    _b.carbon_rms_norm_expand(out, codes, scales, gamma, M, D, _dtype("the output", out), L.handle)
    return out


def _xent_args(x, table, targets):
    import torch
    M, D = _rows("x", x)
    V = _rows("table", table)[0]
    _need("table", table, (V, D), x.dtype)
    _need("targets", targets, (M,), torch.int64)
    return M, D, V, _dtype("x", x)


def linear_cross_entropy_fwd(x, table, targets, ignore_index=-100, reduction="mean", stream=None):
    """(loss, lse): cross entropy of the logits x . table^T against targets.

    x [M, D], table [V, D], targets int64 [M].  loss: fp32, [M] for
    reduction="none", else a scalar (the mean is over the positions that
    count, 0 where there are none); lse: fp32 [M], the rows' log-sum-exp,
    which the gradient takes."""
    import torch
    M, D, V, code = _xent_args(x, table, targets)
    red = _b.REDUCTIONS[reduction]
    L = _Launch(stream)
    losses = L.out((M,), torch.float32, x.device)
    lse = L.out((M,), torch.float32, x.device)
    total = L.out((), torch.float32, x.device) if red else None
    nbytes = _b.carbon_linear_xent_fwd_workspace(M, D, V)
    ws = L.workspace(nbytes, x.device)
    _b.carbon_linear_xent_fwd(losses, total, lse, None, x, table, targets, M, D, V, ignore_index, red, ws, nbytes,
                              code, L.handle)
    return (total if red else losses), lse


def linear_cross_entropy_bwd(grad, x, table, targets, lse, ignore_index=-100, reduction="mean", stream=None):
    """(dx, dtable) from grad (fp32: [M] for reduction="none", else a scalar)."""
    import torch
    M, D, V, code = _xent_args(x, table, targets)
    red = _b.REDUCTIONS[reduction]
    _need("lse", lse, (M,), torch.float32)
    _need("grad", grad, () if red else (M,), torch.float32)
    L = _Launch(stream)
    dx = L.out((M, D), x.dtype, x.device)
    dtable = L.out((V, D), x.dtype, x.device)
    nbytes = _b.carbon_linear_xent_bwd_workspace(M, D, V)
    ws = L.workspace(nbytes, x.device)
    _b.carbon_linear_xent_bwd(dx, dtable, grad, x, table, targets, lse, M, D, V, ignore_index, red, ws, nbytes,
                              code, L.handle)
    return dx, dtable
