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


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("M,D", [(5000, 1), (5000, 3), (4000, 1001), (700, 4099)])
def test_odd_rows_at_any_offset(M, D, dtype):
    """Rows that no 16-byte vector fits give the same bits wherever the tensors
    start: the pieces at both ends that bulk copies cannot take, and what
    follows them in their place."""
    g, dt = gen(M + D), DT[dtype]
    x, res, dy, gamma = (randn(g, *s, dtype=dt) for s in ((M, D), (M, D), (M, D), (D,)))
    want = cg.rms_norm_fwd(x, gamma, res, 1e-5, quantize=True)
    grads = [cg.rms_norm_bwd(dy, gamma, want.rstd, dh=res, recompute=True, **k)
             for k in (dict(h=want.h), dict(codes=want.codes, scales=want.scales))]

    def at(t, offset):
        room = torch.empty(t.numel() + offset, dtype=t.dtype, device="cuda")[offset:].view(t.shape)
        return room.copy_(t)

    for offset in (1, 2, 5):
        r = cg.rms_norm_fwd(at(x, offset), at(gamma, offset), at(res, offset), 1e-5, quantize=True)
        assert all(same_bits(a, b) for a, b in zip(r, want))
        for k, ref in zip((dict(h=at(want.h, offset)), dict(codes=at(want.codes, offset), scales=want.scales)), grads):
            got = cg.rms_norm_bwd(at(dy, offset), at(gamma, offset), want.rstd, dh=at(res, offset), recompute=True, **k)
            assert all(same_bits(a, b) for a, b in zip(got, ref))
    assert status() == 0


@pytest.mark.parametrize("other_stream", [False, True])
def test_rows_without_elements(other_stream):
    """No statistics are left unwritten: the mean of nothing is NaN."""
    stream = torch.cuda.Stream() if other_stream else None
    for _ in range(3):
        junk = torch.full((512,), 7.0, device="cuda")
        torch.cuda.synchronize()
        del junk
        x, gamma = torch.empty(5, 0, device="cuda"), torch.empty(0, device="cuda")
        r = cg.rms_norm_fwd(x, gamma, x, quantize=True, stream=stream)
        torch.cuda.synchronize()
        assert r.y.shape == r.h.shape == r.codes.shape == (5, 0)
        assert bool(torch.isnan(r.rstd).all()) and not bool(r.scales.any())
        dx, dgamma = cg.rms_norm_bwd(x, gamma, r.rstd, h=r.h)
        assert dx.shape == (5, 0) and dgamma.shape == (0,)
    assert status() == 0
