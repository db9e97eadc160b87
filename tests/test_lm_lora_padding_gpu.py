"""Ranks that are no multiple of 16: what pads them takes no part, also where a
row holds an infinity."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import deterministic_invariant_gemm_fwd_gb300 as cg  # noqa: E402
from tests.test_lm_lora_gpu import Case, status  # noqa: E402


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,r", [(5, 8), (5, 16), (300, 24), (130, 72), (300, 128)])
def test_an_infinity_in_a_row(M, r, dtype):
    """All operands positive: the formulas give infinity, not NaN."""
    c = Case(M, 136, 264, 3, r, dtype, M + r, "any")
    for t in (c.x, c.w, c.a, c.b, c.dy, c.scales):
        t.abs_().clamp_(min=2.0 ** -6)
    c.ids[:2] = torch.tensor([1, -1], device="cuda")
    y, u = c.fwd()
    dx, _, _ = c.bwd(u)
    c.x[:2, 3] = math.inf
    c.dy[:2, 5] = math.inf
    y2, u2 = c.fwd()
    dx2, _, _ = c.bwd(u2)
    assert status() == 0
    assert bool((y2[:2] == math.inf).all()) and bool((dx2[:2] == math.inf).all())
    assert torch.equal(y2[2:], y[2:]) and torch.equal(dx2[2:], dx[2:])
    # what pads u is zero
    assert bool((u2[:, :, r:] == 0).all()) and bool((u2[:, 0, :r][0] == math.inf).all())
