"""The C entry points of fine-tuning and scoring as the package exports them give
what the functions of tensors give, and raise the library's errors."""
import array

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import deterministic_invariant_gemm_fwd_gb300 as cg  # noqa: E402
from tests.test_lm_gpu import gen, same_bits, xent_case  # noqa: E402
from tests.test_lm_lora_gpu import Case  # noqa: E402


def f32(*shape):
    return torch.empty(shape, device="cuda")


def room(nbytes):
    assert nbytes >= 0
    return torch.empty(nbytes, dtype=torch.uint8, device="cuda"), nbytes


def test_log_probabilities():
    M, D, V, top = 40, 64, 300, 3
    x, table, t = xent_case(M, D, V, "bf16", 1)
    r = cg.linear_log_probs_fwd(x, table, t, temperature=0.5, top=top)
    logp, entropy, lse, best = f32(M), f32(M), f32(M), f32(M, top)
    ids = torch.empty((M, top), dtype=torch.int64, device="cuda")
    ws, n = room(cg.carbon_linear_logp_fwd_workspace(M, D, V, top))
    cg.carbon_linear_logp_fwd(logp, entropy, lse, ids, best, x, table, t, M, D, V, top, 0.5, -100, ws, n, "bf16")
    assert all(torch.equal(a, b) for a, b in zip((logp, entropy, lse, best, ids), r))
    g = torch.randn(M, generator=gen(2), device="cuda")
    want = cg.linear_log_probs_bwd(g, g, x, table, t, lse, entropy, temperature=0.5)
    dx, dtable = torch.empty_like(x), torch.empty_like(table)
    ws, n = room(cg.carbon_linear_logp_bwd_workspace(M, D, V))
    cg.carbon_linear_logp_bwd(dx, dtable, g, g, x, table, t, lse, entropy, M, D, V, 0.5, -100, ws, n, "bf16")
    assert same_bits(dx, want[0]) and same_bits(dtable, want[1])
    with pytest.raises(cg.CarbonError, match="INVALID_ARG"):
        cg.carbon_linear_logp_fwd(logp, entropy, lse, ids, best, x, table, t, M, D, V, top, 0.5, -100, ws, 8, "bf16")


def test_adapters():
    c = Case(50, 64, 72, 3, 8, "f16", 3)
    y, u = c.fwd()
    M, K, N, n, r = 50, 64, 72, 3, 8
    y2 = torch.empty_like(y)
    u2 = torch.empty(cg.carbon_lora_linear_u_elements(M, r), dtype=y.dtype, device="cuda")
    ws, size = room(cg.carbon_lora_linear_fwd_workspace(M, K, N, n, r))
    cg.carbon_lora_linear_fwd(y2, u2, c.x, c.w, c.bias, c.a, c.b, c.ids, c.scales, M, K, N, n, r, ws, size, "f16")
    assert same_bits(y2, y) and same_bits(u2, u.view(-1))
    dx, da, db = torch.empty_like(c.x), torch.empty_like(c.a), torch.empty_like(c.b)
    ws, size = room(cg.carbon_lora_linear_bwd_workspace(M, K, N, n, r))
    cg.carbon_lora_linear_bwd(dx, da, db, c.dy, c.x, c.w, c.a, c.b, c.ids, c.scales, u2, M, K, N, n, r, ws, size, "f16")
    assert all(same_bits(p, q) for p, q in zip((dx, da, db), c.bwd(u)))


def test_clipping():
    grads = [torch.randn(s, generator=gen(s), device="cuda") for s in (1000, 33)]
    want = [torch.empty_like(g) for g in grads]
    norm = cg.clip_grads(grads, 1.0, out=want)
    out, got = [torch.empty_like(g) for g in grads], f32()
    at, to = (array.array("Q", [t.data_ptr() for t in v]) for v in (grads, out))
    sizes, kinds = array.array("q", [1000, 33]), array.array("i", [0, 0])
    a, b, s, k = (v.buffer_info()[0] for v in (to, at, sizes, kinds))
    ws, n = room(cg.carbon_clip_grads_workspace(s, 2))
    cg.carbon_clip_grads(got, a, b, s, k, 2, 1.0, 1e-6, ws, n)
    assert torch.equal(got, norm) and all(torch.equal(p, q) for p, q in zip(out, want))
