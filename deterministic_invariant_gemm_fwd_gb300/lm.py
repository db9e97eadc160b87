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


def _need(name, t, shape, dtype, device):
    """Raises unless t is a contiguous tensor of this shape and dtype on this
    CUDA device (its index; that of the call's first operand)."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if device < 0 or t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor on the device of the call's other operands")


def _rows(name, t):
    if t.dim() != 2 or not (t.is_cuda and t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous 2-D CUDA tensor")
    return t.shape


class _On:
    """Allocation on a stream that is not the current one: outputs and
    workspace are taken under it, so that neither is memory that the current
    stream still works on.  They belong to that stream, as any tensor made
    under it."""

    def __init__(self, stream):
        self.stream = stream

    def empty(self, shape, dtype, device):
        import torch
        with torch.cuda.stream(self.stream):
            return torch.empty(shape, dtype=dtype, device=device)

    def workspace(self, nbytes, device):
        import torch
        return self.empty(nbytes, torch.uint8, device)


def _begin(t, stream):
    """(stream handle, allocation of outputs, of a workspace) of a call whose
    operands are on t's device."""
    import torch
    device = t.get_device()
    if device != torch.cuda.current_device():
        raise ValueError("the operands must be on the current CUDA device")
    current = torch._C._cuda_getCurrentRawStream(device)
    if stream is not None:
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
        if stream.cuda_stream != current:
            on = _On(stream)
            return stream.cuda_stream, on.empty, on.workspace
    return current, _empty, _workspace


def _empty(shape, dtype, device):
    import torch
    return torch.empty(shape, dtype=dtype, device=device)


def _workspace(nbytes, device):
    import torch
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _bytes(nbytes):
    if nbytes < 0:
        raise ValueError("sizes out of range")
    return nbytes


def _p(t):
    return None if t is None else t.data_ptr()


def embedding_fwd(table, ids, scale=1.0, stream=None):
    """scale * table[ids]: table [V, D], ids int64 of any shape -> [*ids.shape, D]."""
    import torch
    V, D = _rows("table", table)
    shape = ids.shape
    _need("ids", ids, shape, torch.int64, table.get_device())
    code = _dtype("table", table)
    s, empty, _ = _begin(table, stream)
    out = empty((*shape, D), table.dtype, table.device)
    st = _b.lib.carbon_embedding_fwd(out.data_ptr(), table.data_ptr(), ids.data_ptr(), ids.numel(), V, D, scale, code, s)
    if st:
        _b._check(st, "carbon_embedding_fwd")
    return out


def embedding_bwd(dy, ids, num_rows, scale=1.0, padding_idx=-1, accumulate_to=None, stream=None):
    """Gradient of the table: [num_rows, D] from dy [*ids.shape, D].  With
    accumulate_to (a gradient of the same table, e.g. the output layer's) the
    sums are added to it in place and it is returned."""
    import torch
    D, at = dy.shape[-1], dy.get_device()
    shape = ids.shape
    _need("ids", ids, shape, torch.int64, at)
    _need("dy", dy, (*shape, D), dy.dtype, at)
    code = _dtype("dy", dy)
    if accumulate_to is not None:
        _need("accumulate_to", accumulate_to, (num_rows, D), dy.dtype, at)
    s, empty, workspace = _begin(dy, stream)
    out = accumulate_to if accumulate_to is not None else empty((num_rows, D), dy.dtype, dy.device)
    M = ids.numel()
    nbytes = _bytes(_b.lib.carbon_embedding_bwd_workspace(M, num_rows, D))
    ws = workspace(nbytes, dy.device)
    st = _b.lib.carbon_embedding_bwd(out.data_ptr(), dy.data_ptr(), ids.data_ptr(), M, num_rows, D, scale, padding_idx,
                                     0 if accumulate_to is None else 1, ws.data_ptr(), nbytes, code, s)
    if st:
        _b._check(st, "carbon_embedding_bwd")
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
    shape = M, D = _rows("x", x)
    dtype, device, at = x.dtype, x.device, x.get_device()
    code = _dtype("x", x)
    _need("gamma", gamma, (D,), dtype, at)
    if residual is not None:
        _need("residual", residual, shape, dtype, at)
    s, empty, _ = _begin(x, stream)
    h = x if residual is None else empty(shape, dtype, device)
    y = empty(shape, dtype, device)
    rstd = empty(M, torch.float32, device)
    codes = scales = None
    if quantize:
        codes = empty(shape, torch.int8, device)
        scales = empty(M, torch.float32, device)
    st = _b.lib.carbon_rms_norm_fwd(y.data_ptr(), None if residual is None else h.data_ptr(), rstd.data_ptr(), _p(codes),
                                    _p(scales), x.data_ptr(), _p(residual), gamma.data_ptr(), M, D, eps, code, s)
    if st:
        _b._check(st, "carbon_rms_norm_fwd")
    if D == 0:                                   # no elements, no kernel: the mean of nothing, codes of nothing
        with torch.cuda.stream(torch.cuda.ExternalStream(s) if s else torch.cuda.default_stream()):
            rstd.fill_(float("nan"))
            if quantize:
                scales.zero_()
    return RmsNorm(y, h, rstd, codes, scales)


def rms_norm_bwd(dy, gamma, rstd, h=None, codes=None, scales=None, dh=None, recompute=False, stream=None):
    """(dx, dgamma) of rms_norm_fwd from h, or from codes and scales; dx is
    the gradient of x and of the residual.  dh: the gradient that reaches h
    from further on.  recompute=True returns (dx, dgamma, y)."""
    import torch
    shape = M, D = _rows("dy", dy)
    dtype, device, at = dy.dtype, dy.device, dy.get_device()
    code = _dtype("dy", dy)
    _need("gamma", gamma, (D,), dtype, at)
    _need("rstd", rstd, (M,), torch.float32, at)
    if (h is None) == (codes is None) or (codes is None) != (scales is None):
        raise ValueError("give either h, or codes and scales")
    if h is not None:
        _need("h", h, shape, dtype, at)
    else:
        _need("codes", codes, shape, torch.int8, at)
        _need("scales", scales, (M,), torch.float32, at)
    if dh is not None:
        _need("dh", dh, shape, dtype, at)
    s, empty, workspace = _begin(dy, stream)
    dx = empty(shape, dtype, device)
    dgamma = empty(D, dtype, device)
    y = empty(shape, dtype, device) if recompute else None
    nbytes = _bytes(_b.lib.carbon_rms_norm_bwd_workspace(M, D))
    ws = workspace(nbytes, device)
    st = _b.lib.carbon_rms_norm_bwd(dx.data_ptr(), dgamma.data_ptr(), _p(y), dy.data_ptr(), _p(h), _p(codes), _p(scales),
                                    rstd.data_ptr(), gamma.data_ptr(), _p(dh), M, D, ws.data_ptr(), nbytes, code, s)
    if st:
        _b._check(st, "carbon_rms_norm_bwd")
    return (dx, dgamma, y) if recompute else (dx, dgamma)


def rms_norm_expand(codes, scales, gamma=None, dtype=None, stream=None):
    """codes * scales (* gamma) in dtype (gamma's, or bfloat16)."""
    import torch
    shape = M, D = _rows("codes", codes)
    at = codes.get_device()
    _need("codes", codes, shape, torch.int8, at)
    _need("scales", scales, (M,), torch.float32, at)
    dtype = dtype or (gamma.dtype if gamma is not None else torch.bfloat16)
    if gamma is not None:
        _need("gamma", gamma, (D,), dtype, at)
    s, empty, _ = _begin(codes, stream)
    out = empty(shape, dtype, codes.device)
    st = _b.lib.carbon_rms_norm_expand(out.data_ptr(), codes.data_ptr(), scales.data_ptr(), _p(gamma), M, D,
                                       _dtype("the output", out), s)
    if st:
        _b._check(st, "carbon_rms_norm_expand")
    return out


def _xent_args(x, table, targets, reduction):
    import torch
    M, D = _rows("x", x)
    V, at = _rows("table", table)[0], x.get_device()
    _need("table", table, (V, D), x.dtype, at)
    _need("targets", targets, (M,), torch.int64, at)
    if reduction not in _b.REDUCTIONS:
        raise ValueError(f"reduction {reduction!r}; expected one of {sorted(_b.REDUCTIONS)}")
    return M, D, V, _dtype("x", x), _b.REDUCTIONS[reduction]


def linear_cross_entropy_fwd(x, table, targets, ignore_index=-100, reduction="mean", stream=None):
    """(loss, lse): cross entropy of the logits x . table^T against targets.

    x [M, D], table [V, D], targets int64 [M].  loss: fp32, [M] for
    reduction="none", else a scalar (the mean is over the positions that
    count, 0 where there are none); lse: fp32 [M], the rows' log-sum-exp,
    which the gradient takes."""
    import torch
    M, D, V, code, red = _xent_args(x, table, targets, reduction)
    device = x.device
    s, empty, workspace = _begin(x, stream)
    losses = empty(M, torch.float32, device)
    lse = empty(M, torch.float32, device)
    total = empty((), torch.float32, device) if red else None
    nbytes = _bytes(_b.lib.carbon_linear_xent_fwd_workspace(M, D, V))
    ws = workspace(nbytes, device)
    st = _b.lib.carbon_linear_xent_fwd(losses.data_ptr(), _p(total), lse.data_ptr(), None, x.data_ptr(), table.data_ptr(),
                                       targets.data_ptr(), M, D, V, ignore_index, red, ws.data_ptr(), nbytes, code, s)
    if st:
        _b._check(st, "carbon_linear_xent_fwd")
    return (total if red else losses), lse


def linear_cross_entropy_bwd(grad, x, table, targets, lse, ignore_index=-100, reduction="mean", stream=None):
    """(dx, dtable) from grad (fp32: [M] for reduction="none", else a scalar)."""
    import torch
    M, D, V, code, red = _xent_args(x, table, targets, reduction)
    device, at = x.device, x.get_device()
    _need("lse", lse, (M,), torch.float32, at)
    _need("grad", grad, () if red else (M,), torch.float32, at)
    s, empty, workspace = _begin(x, stream)
    dx = empty((M, D), x.dtype, device)
    dtable = empty((V, D), x.dtype, device)
    nbytes = _bytes(_b.lib.carbon_linear_xent_bwd_workspace(M, D, V))
    ws = workspace(nbytes, device)
    st = _b.lib.carbon_linear_xent_bwd(dx.data_ptr(), dtable.data_ptr(), grad.data_ptr(), x.data_ptr(), table.data_ptr(),
                                       targets.data_ptr(), lse.data_ptr(), M, D, V, ignore_index, red, ws.data_ptr(),
                                       nbytes, code, s)
    if st:
        _b._check(st, "carbon_linear_xent_bwd")
    return dx, dtable
