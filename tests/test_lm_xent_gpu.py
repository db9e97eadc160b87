"""The gradient of the output layer's cross entropy on the GPU where its units
depend on each other: sums of dx added in place, small last pieces of the
vocabulary, and gradients that differ from row to row.  References and
tolerances as in test_lm_gpu.py."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import deterministic_invariant_gemm_fwd_gb300 as cg  # noqa: E402
from tests.test_lm_gpu import gen, same_bits, status, within, xent_case, xent_reference  # noqa: E402


def sums_bytes(M, D, V):
    """Bytes of the pieces' sums of dx side by side; above 64 MiB they are added in place."""
    return -(-V // 4096) * (-(-M // 256) * 256) * D * 4


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,D,V", [
    (512, 5120, 32000), (300, 5120, 32000),      # all X units before all T units
    (1, 8192, 50257),
    (4500, 1024, 13000),                         # T units first, pieces one after the other
])
def test_sums_added_in_place(M, D, V, dtype):
    assert sums_bytes(M, D, V) > 64 << 20 and V > 4096
    x, table, t = xent_case(M, D, V, dtype, M + V, kept=1.0)
    g = torch.ones(M, device="cuda")
    _, _, _, eloss, wdx, wdt, edx, edt = xent_reference(x, table, t, g)
    _, lse = cg.linear_cross_entropy_fwd(x, table, t, reduction="none")
    dx, dt = cg.linear_cross_entropy_bwd(g, x, table, t, lse, reduction="none")
    assert status() == 0
    within(dx, wdx, edx)
    within(dt, wdt, edt)
    again = cg.linear_cross_entropy_bwd(g, x, table, t, lse, reduction="none")
    assert same_bits(again[0], dx) and same_bits(again[1], dt)
    # a few rows alone: their sums lie side by side
    for a, b in ((0, 1), (M // 2, M // 2 + 100), (M - 1, M)):
        sl = slice(a, min(b, M))
        rows = sl.stop - sl.start
        if rows < 1 or sums_bytes(rows, D, V) > 64 << 20:
            continue
        part = cg.linear_cross_entropy_bwd(g[sl], x[sl], table, t[sl], lse[sl], reduction="none")[0]
        assert same_bits(part, dx[sl])
    assert status() == 0


@pytest.mark.parametrize("M", [64, 256, 300])
@pytest.mark.parametrize("V", [4160, 4224, 8200])
def test_small_last_piece(M, V):
    """The last piece of the vocabulary is done long before the others, and the
    workspace held NaN: a unit that read G too early would give NaN."""
    D, name = 2048, "bf16"
    x, table, t = xent_case(M, D, V, name, M + V, kept=1.0)
    g = torch.ones(M, device="cuda")
    _, _, _, _, wdx, wdt, edx, edt = xent_reference(x, table, t, g)
    _, lse = cg.linear_cross_entropy_fwd(x, table, t, reduction="none")
    n = cg.carbon_linear_xent_bwd_workspace(M, D, V)
    dx, dt, ws = torch.empty_like(x), torch.empty_like(table), torch.empty(n, dtype=torch.uint8, device="cuda")
    first = None
    for _ in range(5):
        ws.fill_(255)
        cg.carbon_linear_xent_bwd(dx, dt, g, x, table, t, lse, M, D, V, -100, "none", ws, n, name)
        assert status() == 0
        within(dx, wdx, edx)
        within(dt, wdt, edt)
        first = first or (dx.clone(), dt.clone())
        assert same_bits(dx, first[0]) and same_bits(dt, first[1])


@pytest.mark.parametrize("M", [70, 20011])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_gradients_that_are_not_finite(M, dtype):
    """NaN and infinity reach their own row of dx and the table's gradient, and
    no other row of dx."""
    x, table, t = xent_case(M, 64, 300, dtype, M, kept=0.8)
    kept = (t >= 0).nonzero()[:, 0]
    a, b = int(kept[3]), int(kept[-1])
    _, lse = cg.linear_cross_entropy_fwd(x, table, t, reduction="none")

    def bwd(grad, rows=x):
        return cg.linear_cross_entropy_bwd(grad, rows, table, t, lse, reduction="none")

    base = torch.randn(M, generator=gen(1), device="cuda")
    base[a] = base[b] = 0.0
    ref, _ = bwd(base)
    for others in (base, torch.zeros_like(base)):
        want, _ = bwd(others)
        for bad in (float("nan"), float("inf"), float("-inf")):
            g = others.clone()
            g[a], g[b] = bad, float("nan")
            dx, dt = bwd(g)
            assert not bool(torch.isfinite(dx[a]).any()) and bool(torch.isnan(dx[b]).all())
            assert bool(torch.isnan(dt).all())
            rest = torch.ones(M, dtype=torch.bool, device="cuda")
            rest[a] = rest[b] = False
            assert same_bits(dx[rest], want[rest])
    dx, dt = bwd(torch.full_like(base, float("nan")))
    assert bool(torch.isnan(dx[kept]).all()) and not bool(dx[t < 0].any()) and bool(torch.isnan(dt).all())
    # 0 * NaN: a gradient of zero does not hide a row that is not finite
    holed = x.clone()
    holed[a] = float("nan")
    dx, dt = bwd(base, holed)
    assert bool(torch.isnan(dx[a]).all()) and bool(torch.isnan(dt).all())
    # what an ignored position's gradient holds does not matter
    g = base.clone()
    g[t < 0] = float("nan")
    assert same_bits(bwd(g)[0], ref)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_rows_with_gradients_of_different_sizes(dtype):
    """dx of a row does not depend on the gradients of the others, whose
    largest lies outside the part of the batch that is computed again.  fp16: G
    stays in the normal range, whatever the scale."""
    M, D, V = 700, 136, 300 if dtype == "f16" else 9000
    x, table, t = xent_case(M, D, V, dtype, 5, kept=0.9)
    table = table * 0.5
    sign = torch.randint(0, 2, (M,), generator=gen(6), device="cuda") * 2.0 - 1.0
    grad = sign * (0.75 + torch.rand(M, generator=gen(7), device="cuda"))
    lo, hi = int((t >= 0).nonzero()[20, 0]), int((t >= 0).nonzero()[-20, 0])
    grad[lo], grad[hi] = 3.0, -6.7
    if dtype == "f16":
        z = x.double() @ table.double().t()
        assert float(torch.softmax(z, 1).min()) * 0.75 / 8 > 2.0 ** -14 / 2.0 ** 12
    _, lse = cg.linear_cross_entropy_fwd(x, table, t, reduction="none")
    dx, dt = cg.linear_cross_entropy_bwd(grad, x, table, t, lse, reduction="none")
    for a, b in ((0, 1), (13, 14), (100, 229), (0, 513), (lo, M), (lo + 1, hi)):
        sl = slice(a, b)
        part = cg.linear_cross_entropy_bwd(grad[sl], x[sl], table, t[sl], lse[sl], reduction="none")[0]
        assert same_bits(part, dx[sl])
    _, _, _, _, wdx, wdt, edx, edt = xent_reference(x, table, t, grad)
    within(dx, wdx, edx)
    within(dt, wdt, edt)
    # a power of two of every gradient: the same bits, moved
    if dtype == "bf16":
        dx4, dt4 = cg.linear_cross_entropy_bwd(grad * 0.25, x, table, t, lse, reduction="none")
        assert same_bits(dx4 * 4, dx) and same_bits(dt4 * 4, dt)


@pytest.mark.parametrize("reduction", ["none", "sum"])
@pytest.mark.parametrize("size", [2.0 ** -120, 2.0 ** -90, 2.0 ** 100])
def test_gradients_of_extreme_size(size, reduction):
    """The common factor of the gradients neither vanishes nor overflows."""
    M, D, V = 130, 72, 500
    x, table, t = xent_case(M, D, V, "bf16", 3)
    rows = torch.full((M,), size, device="cuda")
    grad = rows if reduction == "none" else rows[0]
    _, lse = cg.linear_cross_entropy_fwd(x, table, t, reduction="none")
    dx, dt = cg.linear_cross_entropy_bwd(grad, x, table, t, lse, reduction=reduction)
    _, _, _, _, wdx, wdt, edx, edt = xent_reference(x, table, t, rows)
    within(dx, wdx, edx)
    within(dt, wdt, edt)
