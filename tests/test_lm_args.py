"""Argument checks of the operators in include/carbon_lm.h on a machine
without a GPU: every bad call is refused before any device is touched, and
the fake pointers below are never dereferenced."""
import pytest

import deterministic_invariant_gemm_fwd_gb300 as cg
from deterministic_invariant_gemm_fwd_gb300 import _binding as b

OK, INVALID, UNSUPPORTED, MISALIGNED, CUDA_ERR = 0, 1, 2, 3, 4
P = 0x1000                       # a fake, 16-byte aligned address
BIG = 1 << 40


def embed_fwd(out=P, table=P, ids=P, M=4, V=5, D=8, scale=1.0, dtype=1):
    return b.lib.carbon_embedding_fwd(out, table, ids, M, V, D, scale, dtype, None)


def embed_bwd(dtable=P, dy=P, ids=P, M=4, V=5, D=8, padding=-1, acc=0, ws=P, nbytes=1 << 30, dtype=1):
    return b.lib.carbon_embedding_bwd(dtable, dy, ids, M, V, D, 1.0, padding, acc, ws, nbytes, dtype, None)


def norm_fwd(y=P, h=P, rstd=P, codes=None, scales=None, x=P, res=None, gamma=P, M=4, D=8, eps=1e-6, dtype=1):
    return b.lib.carbon_rms_norm_fwd(y, h, rstd, codes, scales, x, res, gamma, M, D, eps, dtype, None)


def norm_bwd(dx=P, dgamma=P, y=None, dy=P, h=P, codes=None, scales=None, rstd=P, gamma=P, dh=None, M=4, D=8, ws=P,
             nbytes=1 << 30, dtype=1):
    return b.lib.carbon_rms_norm_bwd(dx, dgamma, y, dy, h, codes, scales, rstd, gamma, dh, M, D, ws, nbytes, dtype,
                                     None)


def expand(out=P, codes=P, scales=P, gamma=None, M=4, D=8, dtype=1):
    return b.lib.carbon_rms_norm_expand(out, codes, scales, gamma, M, D, dtype, None)


def xent_fwd(losses=P, total=P, lse=P, count=None, x=P, table=P, targets=P, M=4, D=8, V=5, red=2, ws=P,
             nbytes=1 << 40, dtype=1):
    return b.lib.carbon_linear_xent_fwd(losses, total, lse, count, x, table, targets, M, D, V, -100, red, ws, nbytes,
                                        dtype, None)


def xent_bwd(dx=P, dtable=P, grad=P, x=P, table=P, targets=P, lse=P, M=4, D=8, V=5, red=2, ws=P, nbytes=1 << 40,
             dtype=1):
    return b.lib.carbon_linear_xent_bwd(dx, dtable, grad, x, table, targets, lse, M, D, V, -100, red, ws, nbytes,
                                        dtype, None)


ALL = [embed_fwd, embed_bwd, norm_fwd, norm_bwd, expand, xent_fwd, xent_bwd]
BAD = [
    (embed_fwd, dict(M=-1)), (embed_fwd, dict(V=-1)), (embed_fwd, dict(D=-8)), (embed_fwd, dict(M=BIG, D=BIG)),
    (embed_fwd, dict(dtype=3)), (embed_fwd, dict(out=None)), (embed_fwd, dict(ids=None)),
    (embed_fwd, dict(table=None)),
    (embed_bwd, dict(M=-1)), (embed_bwd, dict(dtype=-1)), (embed_bwd, dict(dtable=None)),
    (embed_bwd, dict(dy=None)), (embed_bwd, dict(ids=None)), (embed_bwd, dict(padding=5)),
    (embed_bwd, dict(padding=-2)), (embed_bwd, dict(ws=None)), (embed_bwd, dict(ws=P + 4)),
    (embed_bwd, dict(nbytes=15)), (embed_bwd, dict(V=1 << 31)),
    (norm_fwd, dict(M=-1)), (norm_fwd, dict(D=-1)), (norm_fwd, dict(dtype=9)), (norm_fwd, dict(y=None)),
    (norm_fwd, dict(x=None)), (norm_fwd, dict(gamma=None)), (norm_fwd, dict(codes=P)), (norm_fwd, dict(scales=P)),
    (norm_fwd, dict(eps=-1.0)), (norm_fwd, dict(eps=float("nan"))), (norm_fwd, dict(M=1 << 30, D=BIG)),
    (norm_bwd, dict(M=-1)), (norm_bwd, dict(dtype=9)), (norm_bwd, dict(dx=None)), (norm_bwd, dict(dy=None)),
    (norm_bwd, dict(rstd=None)), (norm_bwd, dict(gamma=None)), (norm_bwd, dict(h=None)),
    (norm_bwd, dict(h=None, codes=P)), (norm_bwd, dict(codes=P, scales=P)), (norm_bwd, dict(ws=None)),
    (norm_bwd, dict(nbytes=16)),
    (expand, dict(out=None)), (expand, dict(codes=None)), (expand, dict(scales=None)), (expand, dict(D=-1)),
    (expand, dict(dtype=4)),
    (xent_fwd, dict(M=-1)), (xent_fwd, dict(V=-1)), (xent_fwd, dict(V=0)), (xent_fwd, dict(D=0)),
    (xent_fwd, dict(dtype=7)), (xent_fwd, dict(red=3)), (xent_fwd, dict(red=-1)), (xent_fwd, dict(total=None)),
    (xent_fwd, dict(losses=None)), (xent_fwd, dict(lse=None)), (xent_fwd, dict(x=None)),
    (xent_fwd, dict(table=None)), (xent_fwd, dict(targets=None)), (xent_fwd, dict(ws=None)),
    (xent_fwd, dict(nbytes=16)), (xent_fwd, dict(M=1 << 30)),
    (xent_bwd, dict(M=-1)), (xent_bwd, dict(V=0)), (xent_bwd, dict(red=5)), (xent_bwd, dict(dx=None)),
    (xent_bwd, dict(dtable=None)), (xent_bwd, dict(grad=None)), (xent_bwd, dict(lse=None)),
    (xent_bwd, dict(ws=None)), (xent_bwd, dict(nbytes=16)),
]


@pytest.mark.parametrize("call,args", BAD, ids=lambda v: v.__name__ if callable(v) else str(v))
def test_bad_arguments_are_refused(call, args):
    assert call(**args) == INVALID


@pytest.mark.parametrize("call", [xent_fwd, xent_bwd])
def test_xent_types_and_alignment(call):
    assert call(dtype=0) == UNSUPPORTED
    assert call(D=12) == MISALIGNED
    assert call(x=P + 2) == MISALIGNED
    assert call(table=P + 8) == MISALIGNED
    if call is xent_bwd:
        assert call(dx=P + 8) == MISALIGNED and call(dtable=P + 2) == MISALIGNED


def test_empty_problems_touch_no_device():
    assert embed_fwd(out=None, table=None, ids=None, M=0) == OK
    assert embed_fwd(D=0) == OK
    assert embed_bwd(dtable=None, V=0, padding=-1) == OK
    assert norm_fwd(M=0) == OK and norm_fwd(D=0) == OK
    assert norm_bwd(D=0) == OK and norm_bwd(M=0, dgamma=None) == OK
    assert expand(M=0) == OK
    assert xent_bwd(M=0, V=0) == OK


@pytest.mark.parametrize("call", ALL, ids=lambda f: f.__name__)
def test_injected_launch_failure(call, monkeypatch):
    monkeypatch.setenv("CARBON_FAULT", "launch")
    assert call() == CUDA_ERR
    assert "injected" in b.lib.carbon_last_cuda_error().decode()
    assert call(M=-1) == INVALID


def test_workspace_queries():
    assert b.carbon_embedding_bwd_workspace(-1, 2, 3) == -1
    assert b.carbon_rms_norm_bwd_workspace(3, -1) == -1
    assert b.carbon_linear_xent_fwd_workspace(-1, 8, 8) == -1
    assert b.carbon_linear_xent_bwd_workspace(8, 8, -1) == -1
    # the loss's gradient: bounded per token, far below the logits' 4 bytes per entry
    M, D, V = 8192, 768, 50257
    assert 0 < b.carbon_linear_xent_bwd_workspace(M, D, V) < M * V * 4 // 4
    assert 0 < b.carbon_linear_xent_fwd_workspace(M, D, V) < M * V * 4 // 16


def test_python_refusals():
    import torch
    x, w = torch.zeros(4, 8), torch.zeros(5, 8)
    ids = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError):
        cg.embedding_fwd(w, ids)                                 # not on a GPU
    with pytest.raises(ValueError):
        cg.rms_norm_fwd(x, torch.ones(8))
    with pytest.raises(ValueError):
        cg.linear_cross_entropy_fwd(x, w, ids)
    with pytest.raises(ValueError):
        cg.rms_norm_expand(torch.zeros(4, 8, dtype=torch.int8), torch.zeros(4))


def test_header_from_c(tmp_path):
    """include/carbon_lm.h is plain C: a C99 program links against the library
    and runs on paths that answer without a GPU."""
    import os
    import shutil
    import subprocess
    if shutil.which("gcc") is None:
        pytest.skip("needs gcc")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    exe, libdir = tmp_path / "lm_abi_from_c", os.path.dirname(b.LIB_PATH)
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(root, "include"),
                    os.path.join(root, "tests", "c", "lm_abi_from_c.c"), "-o", str(exe), f"-L{libdir}",
                    "-l:libcarbon_gemm.so", f"-Wl,-rpath,{libdir}"], check=True, capture_output=True, text=True)
    env = dict(os.environ)
    env.pop("CARBON_FAULT", None)
    r = subprocess.run([str(exe)], capture_output=True, text=True, env=env, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stderr


class _Tensor:
    """What the checks of lm.py look at, of a tensor on any device."""

    def __init__(self, shape, dtype, device):
        import torch
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, torch.device("cuda", device)
        self.is_cuda = True

    def dim(self):
        return len(self.shape)

    def get_device(self):
        return self.device.index

    def is_contiguous(self):
        return True

    def data_ptr(self):
        raise AssertionError("the operands reached the library")

    def numel(self):
        return self.shape.numel()


def _calls():
    """(function, its tensors by name as (shape, dtype), the first operand, further arguments)."""
    import torch
    b, f, i, c = torch.bfloat16, torch.float32, torch.int64, torch.int8
    rows = dict(dy=((4, 8), b), gamma=((8,), b), rstd=((4,), f), dh=((4, 8), b))
    loss = dict(x=((4, 8), b), table=((5, 8), b), targets=((4,), i))
    return [
        (cg.embedding_fwd, dict(table=((5, 8), b), ids=((4,), i)), "table", {}),
        (cg.embedding_bwd, dict(dy=((4, 8), b), ids=((4,), i), accumulate_to=((5, 8), b)), "dy", dict(num_rows=5)),
        (cg.rms_norm_fwd, dict(x=((4, 8), b), gamma=((8,), b), residual=((4, 8), b)), "x", {}),
        (cg.rms_norm_bwd, dict(rows, h=((4, 8), b)), "dy", {}),
        (cg.rms_norm_bwd, dict(rows, codes=((4, 8), c), scales=((4,), f)), "dy", {}),
        (cg.rms_norm_expand, dict(codes=((4, 8), c), scales=((4,), f), gamma=((8,), b)), "codes", {}),
        (cg.linear_cross_entropy_fwd, loss, "x", {}),
        (cg.linear_cross_entropy_bwd, dict(loss, lse=((4,), f), grad=((), f)), "x", {}),
    ]


def test_operands_on_different_devices_are_refused(monkeypatch):
    import torch
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0, raising=False)
    for fn, tensors, first, more in _calls():
        for away in tensors:
            args = {k: _Tensor(*v, device=1 if k == away else 0) for k, v in tensors.items()}
            with pytest.raises(ValueError, match="device"):
                fn(**args, **more)


@pytest.mark.parametrize("call", [xent_fwd, xent_bwd])
def test_xent_widest_rows(call, monkeypatch):
    """The launch's limit of column blocks is the widest row: more is refused
    before anything is launched."""
    monkeypatch.setenv("CARBON_FAULT", "launch")
    assert call(D=65535 * 64, M=1, V=1) == CUDA_ERR              # past the checks
    assert call(D=65535 * 64 + 8, M=1, V=1) == INVALID
    query = b.carbon_linear_xent_fwd_workspace if call is xent_fwd else b.carbon_linear_xent_bwd_workspace
    assert query(1, 65535 * 64, 1) > 0 and query(1, 65535 * 64 + 8, 1) == -1


# a pointer that is no multiple of its element's size would fault in a kernel
ODD = [(embed_fwd, "out table"), (embed_bwd, "dtable dy"), (norm_fwd, "y h x res gamma"),
       (norm_bwd, "dx dgamma y dy h gamma dh"), (expand, "out gamma")]
WIDE = [(embed_fwd, dict(ids=8)), (embed_bwd, dict(ids=8)), (norm_fwd, dict(rstd=4)), (norm_bwd, dict(rstd=4)),
        (expand, dict(scales=4)), (xent_fwd, dict(losses=4, total=4, lse=4, count=8, targets=8)),
        (xent_bwd, dict(grad=4, lse=4, targets=8))]


@pytest.mark.parametrize("call,names", ODD, ids=lambda v: v.__name__ if callable(v) else "")
def test_pointers_between_elements_are_refused(call, names, monkeypatch):
    monkeypatch.setenv("CARBON_FAULT", "launch")
    for dtype, size in ((0, 4), (1, 2), (2, 2)):
        for name in names.split():
            assert call(**{name: P + size // 2, "dtype": dtype}) == MISALIGNED, name
            assert call(**{name: P + size, "dtype": dtype}) == CUDA_ERR, name      # elements need no more


@pytest.mark.parametrize("call,names", WIDE, ids=lambda v: v.__name__ if callable(v) else "")
def test_pointers_between_wider_elements_are_refused(call, names, monkeypatch):
    monkeypatch.setenv("CARBON_FAULT", "launch")
    for name, size in names.items():
        assert call(**{name: P + size // 2}) == MISALIGNED, name
        assert call(**{name: P + size}) == CUDA_ERR, name
    if call in (norm_fwd, norm_bwd):
        source = dict(h=None) if call is norm_bwd else {}
        assert call(codes=P + 1, scales=P + 4, **source) == CUDA_ERR
        assert call(codes=P + 1, scales=P + 2, **source) == MISALIGNED
