"""Argument checks of the log probabilities and the low-rank adapters on a
machine without a GPU: every bad call is refused before any device is touched;
the fake addresses are never dereferenced.  Also the order of the tiles that the
alternatives take, on the host."""
import os
import shutil
import subprocess

import pytest

import deterministic_invariant_gemm_fwd_gb300 as cg
from deterministic_invariant_gemm_fwd_gb300 import _binding as b
from tests.test_lm_args import _Tensor

OK, INVALID, UNSUPPORTED, MISALIGNED, CUDA_ERR = 0, 1, 2, 3, 4
P = 0x1000
BIG = 1 << 40
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def logp_fwd(logp=P, ent=P, lse=P, ids=P, best=P, x=P, table=P, tokens=P, M=4, D=8, V=50, top=3, temp=1.0, ws=P,
             nbytes=1 << 40, dtype=1):
    return b.lib.carbon_linear_logp_fwd(logp, ent, lse, ids, best, x, table, tokens, M, D, V, top, temp, -100, ws, nbytes,
                                        dtype, None)


def logp_bwd(dx=P, dtable=P, gl=P, ge=P, x=P, table=P, tokens=P, lse=P, ent=P, M=4, D=8, V=50, temp=1.0, ws=P,
             nbytes=1 << 40, dtype=1):
    return b.lib.carbon_linear_logp_bwd(dx, dtable, gl, ge, x, table, tokens, lse, ent, M, D, V, temp, -100, ws, nbytes,
                                        dtype, None)


def lora_fwd(y=P, u=P, x=P, w=P, bias=P, a=P, bb=P, ids=P, scales=P, M=4, K=8, N=16, n=2, r=8, ws=P, nbytes=1 << 40,
             dtype=1):
    return b.lib.carbon_lora_linear_fwd(y, u, x, w, bias, a, bb, ids, scales, M, K, N, n, r, ws, nbytes, dtype, None)


def lora_bwd(dx=P, da=P, db=P, dy=P, x=P, w=P, a=P, bb=P, ids=P, scales=P, u=P, M=4, K=8, N=16, n=2, r=8, ws=P,
             nbytes=1 << 40, dtype=1):
    return b.lib.carbon_lora_linear_bwd(dx, da, db, dy, x, w, a, bb, ids, scales, u, M, K, N, n, r, ws, nbytes, dtype, None)


ALL = [logp_fwd, logp_bwd, lora_fwd, lora_bwd]
SIZES = [(c, {k: v}) for c, names in ((logp_fwd, "M D V"), (logp_bwd, "M D V"), (lora_fwd, "M K N n r"), (lora_bwd, "M K N n r"))
         for k in names.split() for v in (-1, BIG)]
NULL = [(c, {k: None}) for c, names in
        ((logp_fwd, "logp ent lse ids best x table tokens ws"), (logp_bwd, "dx dtable x table tokens lse ent ws"),
         (lora_fwd, "y u x w a bb ids scales ws"), (lora_bwd, "dy x w a bb ids scales u ws da db"))
        for k in names.split()]
MORE = [(c, d) for c in ALL for d in (dict(dtype=5), dict(dtype=-1), dict(nbytes=8), dict(ws=P + 4))] + [
    (logp_fwd, dict(top=-1)), (logp_fwd, dict(top=29, V=100)), (logp_fwd, dict(top=6, V=5)), (logp_fwd, dict(V=0, top=0)),
    (logp_fwd, dict(D=0)), (logp_bwd, dict(V=0)), (lora_fwd, dict(r=136)), (lora_fwd, dict(K=0)), (lora_fwd, dict(N=0)),
    (lora_fwd, dict(n=0)), (lora_bwd, dict(r=0)), (lora_bwd, dict(dx=None, da=None, db=None)),
] + [(c, dict(temp=t)) for c in (logp_fwd, logp_bwd) for t in (0.0, -1.0, float("nan"), float("inf"), 1e-42, 3.5e-39)]


@pytest.mark.parametrize("call,args", SIZES + NULL + MORE, ids=lambda v: v.__name__ if callable(v) else str(v))
def test_bad_arguments_are_refused(call, args, monkeypatch):
    monkeypatch.setenv("CARBON_FAULT", "launch")
    assert call(**args) == INVALID


def test_arguments_that_may_be_missing(monkeypatch):
    monkeypatch.setenv("CARBON_FAULT", "launch")
    assert logp_fwd(top=0, ids=None, best=None) == CUDA_ERR
    assert logp_bwd(gl=None) == CUDA_ERR and logp_bwd(ge=None, ent=None) == CUDA_ERR
    assert lora_fwd(bias=None) == CUDA_ERR
    assert lora_bwd(da=None, db=None, x=None, u=None) == CUDA_ERR
    assert lora_bwd(dx=None, w=None, a=None) == CUDA_ERR


@pytest.mark.parametrize("call", ALL, ids=lambda f: f.__name__)
def test_injected_launch_failure(call, monkeypatch):
    monkeypatch.setenv("CARBON_FAULT", "launch")
    assert call() == CUDA_ERR and "injected" in b.lib.carbon_last_cuda_error().decode()
    assert call(M=-1) == INVALID


def test_types_and_alignment(monkeypatch):
    monkeypatch.setenv("CARBON_FAULT", "launch")
    for call in ALL:
        assert call(dtype=0) == UNSUPPORTED and call(dtype=2) == CUDA_ERR
    for call, names in ((logp_fwd, "x table"), (logp_bwd, "x table dx dtable"), (lora_fwd, "y u x w a bb"),
                        (lora_bwd, "dx da db dy x w a bb u")):
        for name in names.split():
            assert call(**{name: P + 8}) == MISALIGNED, name
            assert call(**{name: P + 16}) == CUDA_ERR, name
    assert logp_fwd(D=12) == MISALIGNED and logp_bwd(D=12) == MISALIGNED
    for call in (lora_fwd, lora_bwd):
        for name in "KNr":
            assert call(**{name: 12}) == MISALIGNED
    for call, names in ((logp_fwd, dict(logp=4, ent=4, lse=4, best=4, ids=8, tokens=8)),
                        (logp_bwd, dict(gl=4, ge=4, lse=4, ent=4, tokens=8)),
                        (lora_fwd, dict(bias=2, ids=8, scales=4)), (lora_bwd, dict(ids=8, scales=4))):
        for name, size in names.items():
            assert call(**{name: P + size // 2}) == MISALIGNED, name
            assert call(**{name: P + size}) == CUDA_ERR, name


def test_empty_problems_touch_no_device():
    assert logp_bwd(M=0, V=0) == OK
    assert lora_fwd(M=0) == OK and lora_fwd(M=0, y=None, x=None) == OK
    assert lora_bwd(M=0, da=None, db=None) == OK


def test_workspaces():
    for q, n in ((b.carbon_linear_logp_fwd_workspace, 4), (b.carbon_linear_logp_bwd_workspace, 3),
                 (b.carbon_lora_linear_fwd_workspace, 5), (b.carbon_lora_linear_bwd_workspace, 5)):
        for k in range(n):
            assert q(*[-1 if i == k else 8 for i in range(n)]) == -1
    M, D, V = 8192, 768, 50257
    logits = 4 * M * V
    assert b.carbon_linear_logp_fwd_workspace(M, D, V, 0) < logits // 30
    assert b.carbon_linear_logp_fwd_workspace(M, D, V, 8) < logits // 15
    assert b.carbon_linear_logp_bwd_workspace(M, D, V) < logits // 4
    assert b.carbon_lora_linear_u_elements(7, 129) == -1 and b.carbon_lora_linear_u_elements(7, 40) == 7 * 3 * 48
    assert b.carbon_lora_linear_fwd_workspace(M, 768, 2304, 4, 16) < 60 * M


def test_python_refusals():
    import torch
    x, w, ids = torch.zeros(4, 8), torch.zeros(50, 8), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError):
        cg.linear_log_probs_fwd(x, w, ids)                       # not on a GPU
    with pytest.raises(ValueError):
        cg.lora_linear_fwd(x, torch.zeros(8, 16), torch.zeros(2, 8, 8), torch.zeros(2, 8, 16), ids, torch.ones(2))


def _calls():
    import torch
    h, f, i = torch.bfloat16, torch.float32, torch.int64
    logp = dict(x=((4, 8), h), table=((50, 8), h), tokens=((4,), i))
    lora = dict(weight=((8, 16), h), a=((2, 8, 8), h), b=((2, 8, 16), h), adapters=((4,), i), scales=((2,), f))
    return [
        (cg.linear_log_probs_fwd, logp, "x", dict(top=3)),
        (cg.linear_log_probs_bwd, dict(logp, grad_log_probs=((4,), f), grad_entropy=((4,), f), lse=((4,), f), entropy=((4,), f)),
         "x", {}),
        (cg.lora_linear_fwd, dict(lora, x=((4, 8), h), bias=((16,), h)), "x", {}),
        (cg.lora_linear_bwd, dict(lora, dy=((4, 16), h), x=((4, 8), h), u=((4, 3, 16), h)), "dy", {}),
    ]


@pytest.mark.parametrize("what", ["device", "shape", "dtype"])
def test_wrong_operands_are_refused(what, monkeypatch):
    """Each operand in turn on another device, a row longer, of another type."""
    import torch
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0, raising=False)
    for fn, tensors, first, more in _calls():
        for wrong in tensors:
            if wrong == first and what == "dtype":
                continue
            args = {}
            for k, (shape, dtype) in tensors.items():
                if k == wrong and what == "shape":
                    shape = (*shape[:-1], shape[-1] + 8)
                if k == wrong and what == "dtype":
                    dtype = torch.float64
                args[k] = _Tensor(shape, dtype, 1 if k == wrong and what == "device" else 0)
            with pytest.raises((ValueError, TypeError)):
                fn(**args, **more)


def test_wrong_numbers_are_refused(monkeypatch):
    import torch
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    fn, tensors, _, _ = _calls()[0]
    args = {k: _Tensor(*v, 0) for k, v in tensors.items()}
    for more in (dict(top=29), dict(top=-1), dict(top=51), dict(temperature=0.0), dict(temperature=float("nan")),
                 dict(temperature=-2.0), dict(temperature=float("inf"))):
        with pytest.raises(ValueError):
            fn(**args, **more)


def test_header_from_c(tmp_path):
    if shutil.which("gcc") is None:
        pytest.skip("needs gcc")
    exe, libdir = tmp_path / "tune_abi_from_c", os.path.dirname(b.LIB_PATH)
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "include"),
                    os.path.join(ROOT, "tests", "c", "tune_abi_from_c.c"), "-o", str(exe), f"-L{libdir}",
                    "-l:libcarbon_gemm.so", f"-Wl,-rpath,{libdir}"], check=True, capture_output=True, text=True)
    env = dict(os.environ)
    env.pop("CARBON_FAULT", None)
    r = subprocess.run([str(exe)], capture_output=True, text=True, env=env, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stderr


def test_spans_of_tiles(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    exe = str(tmp_path / "xent_spans")
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Wextra", "-Werror", "-I",
                    os.path.join(ROOT, "deterministic_invariant_gemm_fwd_gb300", "csrc"),
                    os.path.join(ROOT, "tests", "c", "xent_spans.cpp"), "-o", exe], check=True, capture_output=True, text=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and r.stdout.strip() == "ok", (r.returncode, r.stderr)


@pytest.mark.parametrize("x_shape, ids_shape", [((4, 16), (4,)), ((2, 3, 8), (6,)), ((2, 3, 8), (3, 2)), ((4, 8), (4, 1)), ((), ())])
def test_shapes_of_the_autograd_functions(x_shape, ids_shape):
    import torch

    from deterministic_invariant_gemm_fwd_gb300 import nn as cnn
    x, ids = torch.zeros(x_shape), torch.zeros(ids_shape, dtype=torch.int64)
    with pytest.raises(ValueError, match="shape"):
        cnn.linear_log_probs(x, torch.zeros(50, 8), ids)
    with pytest.raises(ValueError, match="shape"):
        cnn.top_log_probs(x, torch.zeros(50, 8), ids, 3)
    with pytest.raises(ValueError, match="shape"):
        cnn.lora_linear(x, torch.zeros(8, 16), torch.zeros(2, 8, 8), torch.zeros(2, 8, 16), ids, torch.ones(2))
