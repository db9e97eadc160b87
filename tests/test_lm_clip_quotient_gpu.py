"""Factors of clipping that the quotient max_norm / (norm + eps) does not give."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import deterministic_invariant_gemm_fwd_gb300 as cg  # noqa: E402

TYPES = [torch.float32, torch.bfloat16, torch.float16]


def tensors(*values):
    return [torch.tensor(v, device="cuda").to(t).repeat(40) for t in TYPES for v in values]


def same(a, b):
    return all(torch.equal(p.nan_to_num(7.0, 8.0, 9.0), q.nan_to_num(7.0, 8.0, 9.0)) for p, q in zip(a, b))


@pytest.mark.parametrize("apart", [False, True])
def test_zeros_stay_zeros(apart):
    for max_norm, eps in ((0.0, 0.0), (1.0, 0.0), (math.inf, 0.0), (0.0, 1e-6)):
        grads = tensors([0.0, -0.0, 0.0])
        out = [torch.ones_like(t) for t in grads] if apart else None
        assert float(cg.clip_grads(grads, max_norm, eps=eps, out=out)) == 0.0
        assert all(bool((t == 0).all()) for t in (out or grads))


@pytest.mark.parametrize("apart", [False, True])
def test_an_infinite_bound_scales_nothing(apart):
    for values in ([1.0, math.inf, -2.0], [3.0, 4.0]):
        grads = tensors(values)
        before = [t.clone() for t in grads]
        out = [torch.zeros_like(t) for t in grads] if apart else None
        norm = float(cg.clip_grads(grads, math.inf, out=out))
        assert math.isinf(norm) == (math.inf in values)
        assert same(out or grads, before)
    grads = tensors([1.0, math.nan])
    assert math.isnan(float(cg.clip_grads(grads, math.inf))) and all(bool(t.isnan().all()) for t in grads)


def test_an_infinite_norm_under_a_finite_bound():
    grads = tensors([1.0, math.inf])
    assert math.isinf(float(cg.clip_grads(grads, 2.0)))
    assert all(bool((t[0::2] == 0).all()) and bool(t[1::2].isnan().all()) for t in grads)
