"""The norm on the GPU over its own operands, through the C ABI.  References as in
test_lm_gpu.py."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import deterministic_invariant_gemm_fwd_gb300 as cg  # noqa: E402
from tests.test_lm_gpu import DT, gen, randn, same_bits, status  # noqa: E402


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("D", [768, 1001, 16384, 16392, 20001])
@pytest.mark.parametrize("over", [("x", "residual"), ("residual", "x"), ("x", None), (None, "residual")])
def test_forward_over_its_own_operands(D, dtype, over):
    """y over one of x and residual, the new residual stream over the other:
    the results of separate tensors."""
    M, eps = 37, 1e-5
    g = gen(D)
    x, res, gamma = (randn(g, *s, dtype=DT[dtype]) for s in ((M, D), (M, D), (D,)))
    want = cg.rms_norm_fwd(x, gamma, res, eps, quantize=True)
    own = {"x": x.clone(), "residual": res.clone(), None: None}
    y, h = (torch.empty_like(x) if o is None else own[o] for o in over)
    rstd, codes, scales = torch.empty_like(want.rstd), torch.empty_like(want.codes), torch.empty_like(want.scales)
    cg.carbon_rms_norm_fwd(y, h, rstd, codes, scales, own["x"], own["residual"], gamma, M, D, eps, dtype)
    assert status() == 0
    for a, b in zip((y, h, rstd, codes, scales), want):
        assert same_bits(a, b)
