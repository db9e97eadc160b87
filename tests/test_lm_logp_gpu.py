"""Log probabilities of given tokens, their entropy, alternatives and gradient,
against float64."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import deterministic_invariant_gemm_fwd_gb300 as cg  # noqa: E402
from deterministic_invariant_gemm_fwd_gb300 import nn  # noqa: E402
from tests.test_lm_gpu import E, F16_G, U, gen, same_bits, status, within, xent_case  # noqa: E402

SIZES = [(1, 8, 1), (1, 768, 1000), (7, 64, 129), (130, 72, 257), (64, 320, 5000), (200, 264, 4097), (515, 128, 8200),
         (129, 1096, 700), (300, 64, 20001)]


def reference(x, table, t, temperature):
    """Log probabilities, lse, entropy in float64, and the bounds of what fp32
    products, exponentials and sums cost."""
    M, D = x.shape
    V = table.shape[0]
    z = x.double() @ table.double().t() / temperature
    lse = torch.logsumexp(z, 1)
    keep = (t >= 0) & (t < V)
    at = torch.where(keep, t, 0)
    zt = z[torch.arange(M, device="cuda"), at]
    logp = z - lse[:, None]
    P = torch.exp(logp)
    H = -(P * logp).sum(1)
    ez = D * 2.0 ** -23 * (x.double().abs() @ table.double().abs().t()).amax(1) / temperature
    terms = (16 + math.log2(V)) * 2.0 ** -23
    elp = 2 * ez + terms * (lse.abs() + zt.abs() + 1.0)
    eH = 2 * (H + 1) * ez + terms * (H + 1)
    return keep, at, logp, P, lse, H, zt - lse, ez, elp, eH


def check_forward(x, table, t, temperature, top):
    r = cg.linear_log_probs_fwd(x, table, t, temperature=temperature, top=top)
    assert status() == 0
    keep, at, logp, P, lse, H, lp, ez, elp, eH = reference(x, table, t, temperature)
    zero = torch.zeros_like(lp)
    for got, want, bound in ((r.log_probs, lp, elp), (r.lse, lse, elp), (r.entropy, H, eH)):
        assert bool(((got.double() - torch.where(keep, want, zero)).abs() <= torch.where(keep, bound, zero)).all())
    if top:
        want = torch.sort(logp, dim=1, descending=True, stable=True)
        ids = torch.where(keep[:, None], want.indices[:, :top], -1)
        assert torch.equal(r.top_ids, ids)
        gap = (r.top_log_probs.double() - torch.where(keep[:, None], want.values[:, :top], 0.0)).abs()
        assert bool((gap <= torch.where(keep, elp, zero)[:, None]).all())
    else:
        assert r.top_ids is None and r.top_log_probs is None
    again = cg.linear_log_probs_fwd(x, table, t, temperature=temperature, top=top)
    for a, b in zip(r, again):
        assert a is None or torch.equal(a, b)
    return r


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,D,V", SIZES)
def test_forward(M, D, V, dtype):
    x, table, t = xent_case(M, D, V, dtype, M + D + V)
    for temperature, top in ((1.0, min(5, V)), (0.7, 0), (2.5, min(28, V)), (1.0, min(8, V)), (1.0, min(9, V))):
        r = check_forward(x, table, t, temperature, top)
    # the same results whatever top is
    bare = cg.linear_log_probs_fwd(x, table, t)
    assert all(same_bits(a, b) for a, b in zip(bare[:3], r[:3]))


@pytest.mark.parametrize("D,dtype", [(2048, "bf16"), (4096, "f16")])
def test_mean_error_of_lse(D, dtype):
    # an accumulator that rounds toward zero makes logits smaller by D 2^-30 of
    # themselves on average; put back, less than half of that is left
    x, table, t = xent_case(64, D, 8000, dtype, D)
    z = x.double() @ table.double().t()
    lse = torch.logsumexp(z, 1)
    mean_z = (torch.exp(z - lse[:, None]) * z).sum(1).mean()
    got = cg.linear_log_probs_fwd(x, table, t).lse
    keep = (t >= 0) & (t < 8000)
    assert float((got.double() - lse)[keep].mean().abs()) < 0.5 * D * 2.0 ** -30 * float(mean_z)


@pytest.mark.parametrize("M,V", [(3000, 20000), (9000, 5003), (17000, 300)])
def test_spans_of_several_tiles(M, V):
    x, table, t = xent_case(M, 64, V, "bf16", M, kept=0.9)
    check_forward(x, table, t, 1.0, 8)


@pytest.mark.parametrize("top", [5, 28])
def test_a_position_does_not_depend_on_the_others(top):
    M, D, V = 1100, 128, 9000
    x, table, t = xent_case(M, D, V, "bf16", 5, kept=0.9)
    r = cg.linear_log_probs_fwd(x, table, t, top=top)
    gl, ge = torch.randn(M, generator=gen(2), device="cuda"), torch.full((M,), 0.1, device="cuda")
    dx, _ = cg.linear_log_probs_bwd(gl, ge, x, table, t, r.lse, r.entropy)
    for a, b in ((0, 1), (17, 90), (600, 1100)):
        sl = slice(a, b)
        part = cg.linear_log_probs_fwd(x[sl], table, t[sl], top=top)
        assert all(torch.equal(p, q[sl]) for p, q in zip(part, r))
        d2, _ = cg.linear_log_probs_bwd(gl[sl], ge[sl], x[sl], table, t[sl], part.lse, part.entropy)
        assert same_bits(d2, dx[sl])


# ---- the order of the alternatives -----------------------------------------------

@pytest.mark.parametrize("M", [40, 300])
def test_equal_logits_come_by_entry(M):
    D = 64
    table = torch.randn(50, D, generator=gen(1), device="cuda").bfloat16()
    many = table.repeat(60, 1)                             # 3000 entries, sixty of each
    x = torch.randn(M, D, generator=gen(2), device="cuda").bfloat16()
    t = torch.zeros(M, dtype=torch.long, device="cuda")
    check_forward(x, many, t, 1.0, 28)
    check_forward(torch.zeros_like(x), many, t, 1.0, 20)   # all 3000 equal
    check_forward(x, table[:1].expand(5000, D).contiguous(), t, 1.0, 8)


def test_ascending_and_descending_logits():
    """Every entry passes the threshold, or none after the first."""
    D, V = 64, 30000
    steps = torch.arange(V, device="cuda", dtype=torch.float32)
    table = torch.zeros(V, D, device="cuda")
    table[:, 0], table[:, 1] = steps // 256, steps % 256   # exact in bf16
    x = torch.zeros(300, D, device="cuda")
    x[:, 0], x[:, 1] = 1.0, 2.0 ** -8
    x[1::2] *= -1.0
    t = torch.zeros(300, dtype=torch.long, device="cuda")
    check_forward(x.bfloat16(), table.bfloat16(), t, 1.0, 28)
    check_forward(x.half(), table.half(), t, 0.5, 3)


def test_logits_that_fp32_cannot_tell_apart():
    """Large products that cancel leave differences below fp32's step; the order
    is float64's."""
    D, V, M = 64, 600, 9
    g = gen(4)
    table = torch.zeros(V, D, device="cuda")
    table[:, 0], table[:, 1] = 2.0 ** 20, 2.0 ** 20
    table[:4, 2] = torch.tensor([1.0, 3.0, 2.0, 0.5], device="cuda") * 2.0 ** -9     # lost beside 2^20
    table[4:, 3] = -torch.rand(V - 4, generator=g, device="cuda") - 1.0
    x = torch.ones(M, D, device="cuda")
    x[:, 0] = 1.0 + torch.arange(M, device="cuda") / 16
    x[:, 3] = 64.0
    x, table = x.bfloat16(), table.bfloat16()
    t = torch.zeros(M, dtype=torch.long, device="cuda")
    r = cg.linear_log_probs_fwd(x, table, t, top=4)
    z = x.double() @ table.double().t()
    assert torch.equal(r.top_ids, torch.sort(z, dim=1, descending=True, stable=True).indices[:, :4])
    assert torch.equal(r.top_ids[0], torch.tensor([1, 2, 0, 3], device="cuda"))


def test_infinite_logits_and_nan():
    D, V = 64, 700
    x, table, t = xent_case(6, D, V, "bf16", 8, kept=1.0)
    t[:] = 5
    table[9, 0] = -math.inf                                 # with a positive x[:, 0]: a logit of -infinity
    x[:, 0] = x[:, 0].abs() + 1.0
    r = cg.linear_log_probs_fwd(x, table, t, top=6)
    z = x.double() @ table.double().t()
    keep = torch.arange(V, device="cuda") != 9
    lse = torch.logsumexp(z, 1)
    logp = (z - lse[:, None])[:, keep]
    assert torch.allclose(r.entropy.double(), -(torch.exp(logp) * logp).sum(1), rtol=1e-4, atol=1e-4)
    assert torch.equal(r.top_ids, torch.sort(z, dim=1, descending=True, stable=True).indices[:, :6])
    dx, dt = cg.linear_log_probs_bwd(torch.ones(6, device="cuda"), torch.ones(6, device="cuda"), x, table, t, r.lse, r.entropy)
    assert bool(dt[keep].isfinite().all())
    x[2, 3] = math.nan
    r2 = cg.linear_log_probs_fwd(x, table, t, top=6)
    rest = [0, 1, 3, 4, 5]
    assert all(torch.equal(a[rest], b[rest]) for a, b in zip(r2, r))
    assert bool(r2.log_probs[2].isnan()) and bool(r2.entropy[2].isnan()) and bool((r2.top_ids[2] == -1).all())
    # fewer logits above -infinity than places
    few = torch.zeros(20, D, device="cuda").bfloat16()
    few[3:, 0] = -math.inf
    r3 = cg.linear_log_probs_fwd(torch.ones(2, D, device="cuda").bfloat16(), few, t[:2] * 0, top=5)
    assert torch.equal(r3.top_ids, torch.tensor([[0, 1, 2, -1, -1]] * 2, device="cuda"))
    assert bool((r3.top_log_probs[:, 3:] == -math.inf).all())
    assert status() == 0


# ---- positions that do not count ---------------------------------------------------

def test_ignored_positions():
    M, D, V = 300, 64, 500
    x, table, t = xent_case(M, D, V, "f16", 9, kept=0.5)
    bad = x.clone()
    bad[t < 0] = math.nan
    ref, got = (cg.linear_log_probs_fwd(v, table, t, top=3) for v in (x, bad))
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
    g = torch.randn(M, generator=gen(3), device="cuda")
    a, b = (cg.linear_log_probs_bwd(g, g, v, table, t, ref.lse, ref.entropy) for v in (x, bad))
    assert same_bits(a[0], b[0]) and same_bits(a[1], b[1]) and bool((a[0][t < 0] == 0).all())
    none = torch.full_like(t, -100)
    r = cg.linear_log_probs_fwd(bad, table, none, top=3)
    assert bool((r.log_probs == 0).all()) and bool((r.entropy == 0).all()) and bool((r.top_ids == -1).all())
    dx, dt = cg.linear_log_probs_bwd(g, g, bad, table, none, r.lse, r.entropy)
    assert bool((dx == 0).all()) and bool((dt == 0).all())
    empty = cg.linear_log_probs_fwd(x[:0], table, t[:0], top=3)
    assert empty.log_probs.shape == (0,) and empty.top_ids.shape == (0, 3)
    dx, dt = cg.linear_log_probs_bwd(g[:0], None, x[:0], table, t[:0], empty.lse, empty.entropy)
    assert dx.shape == (0, D) and bool((dt == 0).all())
    assert status() == 0
    wrong = t.clone()
    wrong[0] = V
    r = cg.linear_log_probs_fwd(x, table, wrong, top=3)
    assert cg.carbon_get_device_status() == 7 and float(r.log_probs[0]) == 0.0 and int(r.top_ids[0, 0]) == -1


# ---- gradient ----------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,D,V", SIZES + [(2100, 64, 9000), (17000, 64, 300)])
def test_gradient(M, D, V, dtype):
    x, table, t = xent_case(M, D, V, dtype, M + V)
    g = gen(7)
    for temperature, size in ((1.0, (1.0, 0.1)), (0.7, (1e-6, 1e-4)), (1.3, (0.0, 1.0)), (1.0, (1.0, None))):
        gl = torch.randn(M, generator=g, device="cuda") * size[0]
        ge = None if size[1] is None else torch.randn(M, generator=g, device="cuda") * size[1]
        r = cg.linear_log_probs_fwd(x, table, t, temperature=temperature)
        dx, dt = cg.linear_log_probs_bwd(gl, ge, x, table, t, r.lse, r.entropy, temperature=temperature)
        assert status() == 0
        keep, at, logp, P, lse, H, lp, ez, elp, eH = reference(x, table, t, temperature)
        a = torch.where(keep, gl.double(), 0.0)[:, None]
        e = torch.where(keep, ge.double(), 0.0)[:, None] if ge is not None else torch.zeros_like(a)
        one = torch.zeros_like(P)
        one[torch.arange(M, device="cuda"), at] = 1.0
        c = a + e * (logp + H[:, None])
        G = a * one - P * c
        # P's relative error, the factor's, G's rounding and its spacing near zero
        eP = (2 * ez + elp + 64 * E)[:, None]
        bits = (12 if dtype == "f16" else 32) * math.log(2)
        ec = e.abs() * ((2 * ez + elp + eH)[:, None] + 8 * E * (logp.abs() + bits + H[:, None] + 1)) + 4 * E * a.abs()
        top = float((a.abs() + e.abs() * (math.log(V) + 1)).max())
        gstep = top * (2.0 ** -25 / F16_G if dtype == "f16" else 2.0 ** -133)
        eG = P * (c.abs() * eP + ec) + 4 * E * a.abs() * one + (U[x.dtype] + 4 * E) * G.abs() + gstep * keep[:, None]
        T = temperature
        X, W = x.double(), table.double()
        within(dx, G @ W / T, (eG @ W.abs() + V * 2.0 ** -23 * (G.abs() @ W.abs())) / T)
        within(dt, G.t() @ X / T, (eG.t() @ X.abs() + M * 2.0 ** -23 * (G.abs().t() @ X.abs())) / T)
        again = cg.linear_log_probs_bwd(gl, ge, x, table, t, r.lse, r.entropy, temperature=temperature)
        assert same_bits(again[0], dx) and same_bits(again[1], dt)


def test_entropy_gradient_alone_and_none():
    x, table, t = xent_case(50, 64, 300, "bf16", 3, kept=1.0)
    r = cg.linear_log_probs_fwd(x, table, t)
    g, zero = torch.ones(50, device="cuda"), torch.zeros(50, device="cuda")
    a = cg.linear_log_probs_bwd(None, g, x, table, t, r.lse, r.entropy)
    b = cg.linear_log_probs_bwd(zero, g, x, table, t, r.lse, r.entropy)
    assert same_bits(a[0], b[0]) and same_bits(a[1], b[1])
    dx, dt = cg.linear_log_probs_bwd(None, None, x, table, t, r.lse)
    assert bool((dx == 0).all()) and bool((dt == 0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_gradients_that_are_not_finite(dtype):
    M = 70
    x, table, t = xent_case(M, 64, 300, dtype, M, kept=0.9)
    kept = (t >= 0).nonzero()[:, 0]
    a = int(kept[3])
    r = cg.linear_log_probs_fwd(x, table, t)
    base = torch.randn(M, generator=gen(1), device="cuda")
    other = torch.full((M,), 0.25, device="cuda")
    base[a] = other[a] = 0.0
    ref, _ = cg.linear_log_probs_bwd(base, other, x, table, t, r.lse, r.entropy)
    rest = torch.arange(M, device="cuda") != a
    for bad in (math.nan, math.inf):
        for which in range(2):
            gl, ge = base.clone(), other.clone()
            (gl, ge)[which][a] = bad
            dx, dt = cg.linear_log_probs_bwd(gl, ge, x, table, t, r.lse, r.entropy)
            assert same_bits(dx[rest], ref[rest])
            assert not bool(dx[a].isfinite().any()) and not bool(dt.isfinite().any())


def test_gradient_against_differences():
    M, D, V, T = 33, 64, 300, 0.8
    x, table, t = xent_case(M, D, V, "f16", 13, kept=1.0)
    g = gen(14)
    d, dw = (torch.randn(s, generator=g, device="cuda", dtype=torch.float64) for s in ((M, D), (V, D)))
    gl, ge = torch.randn(M, generator=g, device="cuda"), torch.randn(M, generator=g, device="cuda")

    def f(X, W):
        lp = torch.log_softmax(X @ W.t() / T, 1)
        return (lp.gather(1, t[:, None])[:, 0] * gl).sum() - ((lp.exp() * lp).sum(1) * ge).sum()

    h = 1e-4
    X, W = x.double(), table.double()
    num = (f(X + h * d, W + h * dw) - f(X - h * d, W - h * dw)) / (2 * h)
    r = cg.linear_log_probs_fwd(x, table, t, temperature=T)
    dx, dt = cg.linear_log_probs_bwd(gl, ge, x, table, t, r.lse, r.entropy, temperature=T)
    got = (dx.double() * d).sum() + (dt.double() * dw).sum()
    mag = (dx.double().abs() * d.abs()).sum() + (dt.double().abs() * dw.abs()).sum()
    # two roundings to fp16 (G's entries, the results), each at most half a step of every term
    assert abs(float(num - got)) <= 2 * U[torch.float16] * float(mag) + 1e-3


# ---- streams, graphs, autograd ------------------------------------------------------

def test_another_stream_and_a_graph():
    x, table, t = xent_case(600, 256, 6000, "bf16", 15)
    gl = torch.randn(600, generator=gen(1), device="cuda")
    ref = cg.linear_log_probs_fwd(x, table, t, top=5)
    rdx, rdt = cg.linear_log_probs_bwd(gl, gl, x, table, t, ref.lse, ref.entropy)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    r = cg.linear_log_probs_fwd(x, table, t, top=5, stream=side)
    here = cg.linear_log_probs_fwd(x, table, t, top=5)         # both in flight
    dx, dt = cg.linear_log_probs_bwd(gl, gl, x, table, t, r.lse, r.entropy, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(r, ref)) and all(torch.equal(a, b) for a, b in zip(here, ref))
    assert same_bits(dx, rdx) and same_bits(dt, rdt)
    graph = torch.cuda.CUDAGraph()
    x2 = torch.zeros_like(x)
    with torch.cuda.graph(graph):
        r = cg.linear_log_probs_fwd(x2, table, t, top=5)
        dx, dt = cg.linear_log_probs_bwd(gl, gl, x2, table, t, r.lse, r.entropy)
    x2.copy_(x)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(r, ref)) and same_bits(dx, rdx) and same_bits(dt, rdt)


def test_autograd():
    x, table, t = xent_case(24, 64, 200, "bf16", 16)
    X, W = x.view(4, 6, 64).clone().requires_grad_(), table.clone().requires_grad_()
    lp, ent = nn.linear_log_probs(X, W, t.view(4, 6), temperature=0.9)
    assert lp.shape == ent.shape == (4, 6)
    (lp.sum() * 2.0 + 0.1 * ent.sum()).backward()
    r = cg.linear_log_probs_fwd(x, table, t, temperature=0.9)
    dx, dt = cg.linear_log_probs_bwd(torch.full((24,), 2.0, device="cuda"), torch.full((24,), 0.1, device="cuda"), x,
                                     table, t, r.lse, r.entropy, temperature=0.9)
    assert same_bits(X.grad.view(24, 64), dx) and same_bits(W.grad, dt)
    # only one of the outputs goes on; no second derivatives
    X.grad = None
    nn.linear_log_probs(X, W, t.view(4, 6))[1].sum().backward()
    r = cg.linear_log_probs_fwd(x, table, t)
    want = cg.linear_log_probs_bwd(None, torch.ones(24, device="cuda"), x, table, t, r.lse, r.entropy)[0]
    assert same_bits(X.grad.view(24, 64), want)
    (gx,) = torch.autograd.grad(nn.linear_log_probs(X, W, t.view(4, 6))[0].sum(), X, create_graph=True)
    with pytest.raises(RuntimeError, match="no derivative"):
        gx.sum().backward()
    with torch.no_grad():
        s = nn.top_log_probs(X, W, t.view(4, 6), top=3)
    assert s.top_ids.shape == (4, 6, 3) and s.log_probs.shape == (4, 6)
    with pytest.raises(ValueError):
        nn.linear_log_probs(X, W, t)
