"""Argument checks of gradient clipping on a machine without a GPU: refused
before any device is touched; the fake addresses are never dereferenced."""
import array

import pytest

from deterministic_invariant_gemm_fwd_gb300 import _binding as b

OK, INVALID, MISALIGNED, CUDA_ERR = 0, 1, 3, 4
P = 0x100000


def clip(norm=P, out=(P + 0x1000, P + 0x2000), grads=(P + 0x1000, P + 0x2000), sizes=(10, 20), dtypes=(0, 1), count=2,
         max_norm=1.0, eps=1e-6, ws=P + 0x8000, nbytes=1 << 20):
    def at(code, v):
        if v is None:
            return None, None
        a = array.array(code, v)
        return a, a.buffer_info()[0]
    keep = [at("Q", out), at("Q", grads), at("q", sizes), at("i", dtypes)]
    o, g, s, d = (k[1] for k in keep)
    return b.lib.carbon_clip_grads(norm, o, g, s, d, count, max_norm, eps, ws, nbytes, None)


BAD = [dict(count=-1), dict(sizes=None), dict(grads=None), dict(dtypes=None), dict(norm=None, out=None),
       dict(sizes=(-1, 4)), dict(sizes=(1 << 50, 4)), dict(dtypes=(0, 3)), dict(dtypes=(-1, 1)), dict(max_norm=-1.0),
       dict(max_norm=float("nan")), dict(eps=-1.0), dict(ws=None), dict(ws=P + 8), dict(nbytes=15),
       dict(grads=(0, P + 0x2000)), dict(out=(P + 0x1000, 0)),
       dict(grads=(P + 0x1000, P + 0x1000), out=(P + 0x1000, P + 0x1000)),          # the same tensor twice
       dict(out=(P + 0x1000, P + 0x1020)), dict(out=(P + 0x2010, P + 0x3000)), dict(out=(P + 0x1004, P + 0x2000)),
       dict(grads=(P, P + 0x100), out=(P + 0x80, P + 0x200), sizes=(100, 3))]


@pytest.mark.parametrize("args", BAD, ids=str)
def test_bad_arguments_are_refused(args, monkeypatch):
    monkeypatch.setenv("CARBON_FAULT", "launch")
    assert clip(**args) == INVALID


def test_accepted_calls_reach_the_launch(monkeypatch):
    monkeypatch.setenv("CARBON_FAULT", "launch")
    for args in (dict(), dict(out=None), dict(out=(P + 0x5000, P + 0x6000)), dict(norm=None), dict(sizes=(0, 5)),
                 dict(grads=(P + 0x1000, P + 0x1004), out=(P + 0x5000, P + 0x6000)),        # only read twice
                 dict(grads=(P + 0x1000, P + 0x1028), out=(P + 0x1000, P + 0x1028)),        # one behind the other
                 dict(out=None, max_norm=-1.0), dict(max_norm=float("inf"))):
        assert clip(**args) == CUDA_ERR, args
        assert "injected" in b.lib.carbon_last_cuda_error().decode()


def test_alignment(monkeypatch):
    monkeypatch.setenv("CARBON_FAULT", "launch")
    assert clip(norm=P + 2) == MISALIGNED
    assert clip(grads=(P + 0x1002, P + 0x2000), out=None) == MISALIGNED
    assert clip(out=(P + 0x1000, P + 0x2001)) == MISALIGNED
    assert clip(grads=(P + 0x1004, P + 0x2002), out=(P + 0x5004, P + 0x6002)) == CUDA_ERR


def test_nothing_to_do_touches_no_device():
    assert clip(norm=None, sizes=(0, 0)) == OK
    assert clip(norm=None, out=(0, 0), grads=(0, 0), sizes=(0, 0), count=0, ws=None, nbytes=0) == OK


def test_workspace():
    one = array.array("q", [1] * 3)
    assert b.carbon_clip_grads_workspace(one.buffer_info()[0], 3) >= 24
    big = array.array("q", [1 << 40])
    assert b.carbon_clip_grads_workspace(big.buffer_info()[0], 1) <= (64 << 10) + 64
    assert b.carbon_clip_grads_workspace(None, 2) == -1
    bad = array.array("q", [-1])
    assert b.carbon_clip_grads_workspace(bad.buffer_info()[0], 1) == -1


def test_python_refusals():
    import torch

    import deterministic_invariant_gemm_fwd_gb300 as cg
    from deterministic_invariant_gemm_fwd_gb300 import nn
    with pytest.raises(ValueError):
        cg.clip_grads([torch.zeros(4)], 1.0)                 # not on a GPU
    with pytest.raises(ValueError):
        cg.clip_grads([torch.zeros(4)], float("nan"))
    with pytest.raises(TypeError):
        cg.grad_norm([torch.zeros(4, dtype=torch.int64)])
    assert float(nn.clip_grad_norm_([torch.nn.Parameter(torch.zeros(3))], 1.0)) == 0.0
