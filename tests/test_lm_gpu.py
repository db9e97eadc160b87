"""The operators around the linear layers on the GPU against plain float64
implementations: token embedding, RMS norm with its 8-bit checkpoint, and the
output layer's softmax cross entropy, forward and backward.

Tolerances come from rounding-error bounds of the definitions: u(T) is the
unit roundoff of the output type, 2^-24 that of the fp32 sums, n terms added
in any order cost at most n * 2^-24 of the sum of magnitudes."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import deterministic_invariant_gemm_fwd_gb300 as cg  # noqa: E402
from deterministic_invariant_gemm_fwd_gb300 import nn as cnn  # noqa: E402

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
# half the spacing of the smallest values of the type
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25}
E = 2.0 ** -24
F16_G = 2.0 ** 12                # G's scale in fp16


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, dtype, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def status():
    return cg.carbon_get_device_status()


def within(got, want, slack):
    """|got - want| <= slack + one rounding of want to got's type, elementwise."""
    u, tiny = U[got.dtype], TINY[got.dtype]
    lim = slack + u * (want.abs() + slack) + tiny
    bad = (got.double() - want).abs() > lim
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()}, worst ratio " \
        f"{float(((got.double() - want).abs() / lim).max())}"


def same_bits(a, b):
    a, b = a.contiguous(), b.contiguous()
    return a.dtype == b.dtype and a.shape == b.shape and torch.equal(a.view(-1).view(torch.uint8),
                                                                     b.view(-1).view(torch.uint8))


# ---- embedding ---------------------------------------------------------------------

EMBED = [(1, 1, 1), (1, 5, 8), (3, 2, 7), (33, 100, 24), (257, 1000, 515), (700, 31, 136), (1025, 513, 72),
         (5000, 50257, 64), (70000, 300, 16)]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("M,V,D", EMBED)
def test_embedding(M, V, D, dtype):
    g, dt = gen(M + V), DT[dtype]
    table = randn(g, V, D, dtype=dt)
    # squares crowd the low ids: long runs of one token
    ids = (torch.rand(M, generator=g, device="cuda") ** 2 * V).long().clamp_(max=V - 1)
    scale = math.sqrt(D)
    s32 = float(torch.tensor(scale, dtype=torch.float32))
    out = cg.embedding_fwd(table, ids, scale)
    within(out, table.double()[ids] * s32, E * (table.double()[ids] * s32).abs())
    dy = randn(g, M, D, dtype=dt)
    got = cg.embedding_bwd(dy, ids, V, scale)
    want = torch.zeros(V, D, dtype=torch.float64, device="cuda").index_add_(0, ids, dy.double()) * s32
    mag = torch.zeros(V, D, dtype=torch.float64, device="cuda").index_add_(0, ids, dy.double().abs()) * s32
    n = torch.bincount(ids, minlength=V).double()[:, None]
    within(got, want, (n + 2) * E * mag)
    assert same_bits(got, cg.embedding_bwd(dy, ids, V, scale))
    # onto a gradient that is there
    base = randn(g, V, D, dtype=dt)
    acc = base.clone()
    assert cg.embedding_bwd(dy, ids, V, scale, accumulate_to=acc) is acc
    within(acc, base.double() + want, (n + 3) * E * (mag + base.double().abs()))
    untouched = (n == 0).squeeze(1)
    assert same_bits(acc[untouched], base[untouched])
    assert status() == 0


def test_embedding_one_token_everywhere():
    M, D = 5003, 40
    dy = randn(gen(1), M, D, dtype=torch.bfloat16)
    ids = torch.full((M,), 7, device="cuda")
    got = cg.embedding_bwd(dy, ids, 9)
    within(got[7], dy.double().sum(0), M * E * dy.double().abs().sum(0))
    assert not bool(got[:7].any()) and not bool(got[8:].any())


def test_embedding_padding_and_ids_outside_the_table():
    V, D = 11, 24
    table = randn(gen(2), V, D, dtype=torch.float16)
    ids = torch.tensor([[3, -1, 3], [V, 5, 2 ** 40]], device="cuda")
    out = cg.embedding_fwd(table, ids)
    assert status() == 7 and status() == 0
    ok = (ids >= 0) & (ids < V)
    assert torch.equal(out[ok], table[ids[ok]]) and not bool(out[~ok].any())
    dy = randn(gen(3), 2, 3, D, dtype=torch.float16)
    dy[~ok] = float("nan")                       # left out, whatever it holds
    got = cg.embedding_bwd(dy, ids, V, padding_idx=5)
    assert status() == 7 and status() == 0
    want = torch.zeros(V, D, dtype=torch.float64, device="cuda")
    want[3] = dy[0, 0].double() + dy[0, 2].double()
    within(got, want, 2 * E * want.abs())
    # a padded id alone is no error
    cg.embedding_bwd(dy[:, 1:2].contiguous(), torch.full((2, 1), 5, device="cuda"), V, padding_idx=5)
    assert status() == 0


def test_embedding_without_tokens():
    dy = torch.empty(0, 16, device="cuda")
    ids = torch.empty(0, dtype=torch.int64, device="cuda")
    assert cg.embedding_fwd(torch.zeros(3, 16, device="cuda"), ids).shape == (0, 16)
    assert not bool(cg.embedding_bwd(dy, ids, 6).any())
    keep = torch.ones(6, 16, device="cuda")
    assert bool((cg.embedding_bwd(dy, ids, 6, accumulate_to=keep) == 1).all())


def test_embedding_rows_past_32_bits():
    """Element offsets beyond 2^32 in the table and in its gradient."""
    V, D = 2 ** 23 + 5, 520
    table = torch.zeros(V, D, dtype=torch.bfloat16, device="cuda")
    ids = torch.tensor([V - 1, 0, V - 1, V - 2], device="cuda")
    table[ids] = randn(gen(4), 4, D, dtype=torch.bfloat16)
    assert torch.equal(cg.embedding_fwd(table, ids), table[ids])
    dy = randn(gen(5), 4, D, dtype=torch.bfloat16)
    got = cg.embedding_bwd(dy, ids, V)
    within(got[V - 1], dy[0].double() + dy[2].double(), 2 * E * (dy[0].double().abs() + dy[2].double().abs()))
    assert torch.equal(got[V - 2], dy[3]) and torch.equal(got[0], dy[1])
    assert int(got.ne(0).any(1).sum()) == 3


# ---- norm ----------------------------------------------------------------------------

NORM = [(1, 1), (1, 768), (3, 5), (2, 256), (5, 257), (9, 515), (33, 1024), (7, 1032), (4, 2056), (650, 96), (5, 4096),
        (3, 4104), (2, 16384), (3, 16392), (2, 20001), (1300, 72)]


def norm_reference(x, res, gamma, eps):
    h = x.double() + (res.double() if res is not None else 0.0)
    rstd = 1.0 / torch.sqrt((h * h).mean(1) + eps)
    n = h * rstd[:, None]
    return h, rstd, n, n * gamma.double()


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("M,D", NORM)
def test_rms_norm_forward(M, D, dtype):
    g, dt = gen(M * 31 + D), DT[dtype]
    x, res = randn(g, M, D, dtype=dt), randn(g, M, D, dtype=dt, std=3.0)
    gamma = randn(g, D, dtype=dt)
    eps = 1e-5
    rel = (D + 16) * E                           # of rstd: a sum of D squares, a division, a root
    for residual in (res, None):
        r = cg.rms_norm_fwd(x, gamma, residual, eps, quantize=True)
        h, rstd, n, y = norm_reference(x, residual, gamma, float(torch.tensor(eps, dtype=torch.float32)))
        within(r.rstd, rstd, rel * rstd)
        within(r.y, y, (rel + 4 * E) * y.abs())
        if residual is None:
            assert r.h is x
        else:
            within(r.h, h, E * h.abs())
        # the checkpoint: scale = max / 127, every value within half a step
        top = n.abs().amax(1)
        within(r.scales, top / 127.0, (rel + 4 * E) * top / 127.0)
        s = r.scales.double()[:, None]
        half = s * (0.5 + 127 * (rel + 8 * E)) + s * 127 * 8 * E
        assert bool(((r.codes.double() * s - n).abs() <= half).all())
        assert int(r.codes.abs().amax()) == 127
        back = cg.rms_norm_expand(r.codes, r.scales, gamma)
        want = r.codes.double() * s * gamma.double()
        within(back, want, 2 * E * want.abs())
        plain = cg.rms_norm_fwd(x, gamma, residual, eps)
        assert same_bits(plain.y, r.y) and plain.codes is None
    # a row's result does not depend on the others
    one = cg.rms_norm_fwd(x[M - 1:].contiguous(), gamma, res[M - 1:].contiguous(), eps, quantize=True)
    full = cg.rms_norm_fwd(x, gamma, res, eps, quantize=True)
    assert all(same_bits(a[-1:], b) for a, b in zip(full, one))
    assert status() == 0


@pytest.mark.parametrize("source", ["h", "codes"])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("M,D", NORM)
def test_rms_norm_backward(M, D, dtype, source):
    g, dt = gen(M * 17 + D), DT[dtype]
    h, dy, dh = (randn(g, M, D, dtype=dt, std=s) for s in (2.0, 1.0, 0.5))
    gamma = randn(g, D, dtype=dt)
    rstd = torch.rsqrt(h.float().square().mean(1) + 1e-5)
    kw = {"h": h}
    n = h.double() * rstd.double()[:, None]
    if source == "codes":
        r = cg.rms_norm_fwd(h, gamma, None, 1e-5, quantize=True)
        kw = {"codes": r.codes, "scales": r.scales}
        n = r.codes.double() * r.scales.double()[:, None]
    gdy = gamma.double() * dy.double()
    dot, dotmag = (gdy * n).mean(1, keepdim=True), (gdy * n).abs().mean(1, keepdim=True)
    rs = rstd.double()[:, None]
    for extra in (dh, None):
        add = extra.double() if extra is not None else torch.zeros_like(n)
        dx, dgamma, y = cg.rms_norm_bwd(dy, gamma, rstd, dh=extra, recompute=True, **kw)
        want = rs * (gdy - n * dot) + add
        slack = rs * (4 * E * gdy.abs() + n.abs() * ((D + 12) * E * dotmag + 6 * E * dot.abs())) + 2 * E * (
            add.abs() + want.abs())
        within(dx, want, slack)
        mag = (dy.double() * n).abs().sum(0)
        within(dgamma, (dy.double() * n).sum(0), (M + 4) * E * mag)
        within(y, n * gamma.double(), 3 * E * (n * gamma.double()).abs())
        two = cg.rms_norm_bwd(dy, gamma, rstd, dh=extra, **kw)
        assert same_bits(two[0], dx) and same_bits(two[1], dgamma)
    last = {k: v[M - 1:].contiguous() for k, v in kw.items()}
    one = cg.rms_norm_bwd(dy[M - 1:].contiguous(), gamma, rstd[M - 1:].contiguous(), **last)
    assert same_bits(one[0], cg.rms_norm_bwd(dy, gamma, rstd, **kw)[0][M - 1:])
    assert status() == 0


def test_rms_norm_unaligned_operands():
    """Contiguous tensors that do not start on a 16-byte boundary."""
    M, D, dt = 6, 768, torch.bfloat16

    def odd(*shape, dtype=dt):
        n = math.prod(shape)
        return torch.empty(n + 1, dtype=dtype, device="cuda")[1:].view(*shape)

    g = gen(9)
    x, res, gamma = odd(M, D), odd(M, D), odd(D)
    for t in (x, res, gamma):
        t.copy_(randn(g, *t.shape, dtype=dt))
    a = cg.rms_norm_fwd(x, gamma, res, 1e-5, quantize=True)
    h, rstd, n, y = norm_reference(x, res, gamma, 1e-5)
    within(a.y, y, (D + 24) * E * y.abs())
    codes = odd(M, D, dtype=torch.int8)
    codes.copy_(a.codes)
    ref = cg.rms_norm_bwd(a.y, gamma, a.rstd, codes=a.codes, scales=a.scales)
    got = cg.rms_norm_bwd(a.y, gamma, a.rstd, codes=codes, scales=a.scales)
    within(got[0], ref[0].double(), 2.0 ** -7 * ref[0].double().abs() + 1e-6)
    assert same_bits(cg.rms_norm_expand(codes, a.scales, gamma), cg.rms_norm_expand(a.codes, a.scales, gamma))
    ids = torch.tensor([2, 0, 2], device="cuda")
    assert torch.equal(cg.embedding_fwd(x, ids), x[ids])
    within(cg.embedding_bwd(odd(3, D).copy_(x[:3]), ids, 4)[2], x[0].double() + x[2].double(),
           2 * E * (x[0].double().abs() + x[2].double().abs()))


def test_rms_norm_zero_rows_and_values_that_are_not_finite():
    D = 40
    x = randn(gen(7), 6, D, dtype=torch.float32)
    x[0] = 0.0
    x[1, 3], x[2, 5], x[3, 7] = float("nan"), float("inf"), float("-inf")
    x[4] *= 1e-38                                 # far below eps
    gamma = torch.ones(D, device="cuda")
    r = cg.rms_norm_fwd(x, gamma, None, 1e-5, quantize=True)
    assert not bool(r.y[0].any()) and float(r.scales[0]) == 0.0 and not bool(r.codes[0].any())
    for m in (1, 2, 3):
        assert math.isnan(float(r.scales[m])) and not bool(r.codes[m].any())
        assert bool(torch.isnan(cg.rms_norm_expand(r.codes, r.scales, gamma)[m]).all())
    assert float(r.scales[4]) == 0.0 and not bool(r.codes[4].any())
    clean = cg.rms_norm_fwd(x[5:].contiguous(), gamma, None, 1e-5, quantize=True)
    assert same_bits(r.y[5:], clean.y) and same_bits(r.codes[5:], clean.codes)
    # eps = 0 and a zero row: 0 * inf
    assert bool(torch.isnan(cg.rms_norm_fwd(x[:1].contiguous(), gamma, None, 0.0).y).all())


def test_rms_norm_without_rows():
    x, gamma = torch.empty(0, 24, device="cuda"), torch.ones(24, device="cuda")
    r = cg.rms_norm_fwd(x, gamma, x, quantize=True)
    assert r.y.shape == (0, 24) and r.codes.shape == (0, 24)
    dx, dgamma = cg.rms_norm_bwd(x, gamma, r.rstd, h=r.h)
    assert dx.shape == (0, 24) and not bool(dgamma.any())
    assert cg.rms_norm_expand(r.codes, r.scales, gamma).shape == (0, 24)
    assert status() == 0


def test_rms_norm_gradient_over_its_own_operand():
    """dx may be dh's memory (the C call); also with odd rows, whose bulk
    copies reach into their neighbours."""
    M, D = 700, 515
    g = gen(31)
    h, dy, dh = (randn(g, M, D, dtype=torch.bfloat16) for _ in range(3))
    gamma = randn(g, D, dtype=torch.bfloat16)
    r = cg.rms_norm_fwd(h, gamma)
    ref, dgamma = cg.rms_norm_bwd(dy, gamma, r.rstd, h=h, dh=dh)
    n = cg.carbon_rms_norm_bwd_workspace(M, D)
    ws, dg = torch.empty(n, dtype=torch.uint8, device="cuda"), torch.empty_like(gamma)
    both = dh.clone()
    cg.carbon_rms_norm_bwd(both, dg, None, dy, h, None, None, r.rstd, gamma, both, M, D, ws, n, "bf16")
    assert same_bits(both, ref) and same_bits(dg, dgamma)


def test_rms_norm_gradient_against_differences():
    """sum(y * w) and the residual stream's sum(h * v), in float64 central
    differences along random directions."""
    M, D, eps = 5, 48, 1e-5
    g = gen(11)
    x, res, gamma, w, v = (randn(g, M if i != 2 else 1, D, dtype=torch.float32) for i in range(5))
    gamma = gamma[0].contiguous()
    r = cg.rms_norm_fwd(x, gamma, res, eps)
    dx, dgamma = cg.rms_norm_bwd(w, gamma, r.rstd, h=r.h, dh=v)

    def f(x64, g64):
        h = x64 + res.double()
        return ((h / torch.sqrt((h * h).mean(1, keepdim=True) + eps) * g64) * w.double()).sum() + (h * v.double()).sum()

    d, dg = (torch.randn(s, generator=g, device="cuda", dtype=torch.float64) for s in ((M, D), (D,)))
    t = 1e-5
    num = (f(x.double() + t * d, gamma.double() + t * dg) - f(x.double() - t * d, gamma.double() - t * dg)) / (2 * t)
    got = (dx.double() * d).sum() + (dgamma.double() * dg).sum()
    mag = (dx.double() * d).abs().sum() + (dgamma.double() * dg).abs().sum()
    # fp32 results: (D + 40) roundings of each term; differences: t^2 and 1e-16 / t
    assert abs(float(num - got)) <= float(mag) * (D + 40) * E + 1e-6


# ---- cross entropy -------------------------------------------------------------------

XENT = [(1, 8, 1), (1, 768, 1000), (7, 64, 129), (130, 72, 257), (64, 320, 5000), (200, 264, 4097), (515, 128, 8200),
        (129, 1096, 700), (300, 64, 20001)]


def xent_case(M, D, V, dtype, seed, kept=0.75):
    g, dt = gen(seed), DT[dtype]
    x, table = randn(g, M, D, dtype=dt), randn(g, V, D, dtype=dt, std=2.0 / math.sqrt(D))
    t = torch.randint(0, V, (M,), generator=g, device="cuda")
    t[torch.rand(M, generator=g, device="cuda") >= kept] = -100
    if M == 1:
        t[0] = V // 2
    return x, table, t


def xent_reference(x, table, t, grad_rows):
    """Losses, lse and gradients in float64 for gradients per row, and the
    bound of what fp32 products and a rounded G cost."""
    M, D = x.shape
    u = U[x.dtype]
    X, W = x.double(), table.double()
    z = X @ W.t()
    lse = torch.logsumexp(z, 1)
    keep = (t >= 0) & (t < table.shape[0])
    at = torch.where(keep, t, 0)
    row = torch.arange(M, device="cuda")
    loss = torch.where(keep, lse - z[row, at], 0.0)
    # a sum of D products into an fp32 accumulator that may truncate, twice (z and lse), and the exponentials
    ez = (2 * D * 2.0 ** -23) * (X.abs() @ W.abs().t()).amax(1)
    eloss = ez + (16 + math.log2(table.shape[0])) * 2 * E * (lse.abs() + z[row, at].abs() + 1.0)
    P = torch.exp(z - lse[:, None])
    one = torch.zeros_like(P)
    one[row, at] = 1.0
    r = torch.where(keep, grad_rows.double(), 0.0)[:, None]
    G = (P - one) * r
    # G's relative error through P, its rounding (twice where rows differ), its spacing near zero
    top = float(r.abs().max())
    gstep = top * (2.0 ** -25 / F16_G if x.dtype == torch.float16 else 2.0 ** -133)
    eG = P * r.abs() * (2 * ez[:, None] + eloss[:, None] + 64 * E) + (u + 4 * E) * G.abs() + gstep * (r != 0)
    dx, dt = G @ W, G.t() @ X
    V = table.shape[0]
    edx = eG @ W.abs() + V * 2.0 ** -23 * (G.abs() @ W.abs())
    edt = eG.t() @ X.abs() + M * 2.0 ** -23 * (G.abs().t() @ X.abs())
    return loss, lse, keep, eloss, dx, dt, edx, edt


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,D,V", XENT)
def test_cross_entropy(M, D, V, dtype):
    x, table, t = xent_case(M, D, V, dtype, M + D + V)
    grad = torch.randn(M, generator=gen(3), device="cuda")
    loss, lse, keep, eloss, dx, dt, edx, edt = xent_reference(x, table, t, grad)
    got, got_lse = cg.linear_cross_entropy_fwd(x, table, t, reduction="none")
    within(got, loss, eloss)
    within(got_lse, torch.where(keep, lse, 0.0), eloss)
    assert not bool(got[~keep].any()) and not bool(got_lse[~keep].any())
    gdx, gdt = cg.linear_cross_entropy_bwd(grad, x, table, t, got_lse, reduction="none")
    within(gdx, dx, edx)
    within(gdt, dt, edt)
    assert not bool(gdx[~keep].any())
    again = cg.linear_cross_entropy_bwd(grad, x, table, t, got_lse, reduction="none")
    assert same_bits(again[0], gdx) and same_bits(again[1], gdt)
    # sums and means
    count = max(1, int(keep.sum()))
    for red, div in (("sum", 1), ("mean", count)):
        total, _ = cg.linear_cross_entropy_fwd(x, table, t, reduction=red)
        want = loss.sum() / div
        within(total, want, eloss.sum() / div)
        g0 = torch.tensor(0.75, device="cuda")
        dx, dt, edx, edt = xent_reference(x, table, t, torch.full((M,), 0.75 / div, device="cuda", dtype=torch.float64))[4:]
        sdx, sdt = cg.linear_cross_entropy_bwd(g0, x, table, t, got_lse, reduction=red)
        within(sdx, dx, edx + 2 * E * dx.abs())
        within(sdt, dt, edt + 2 * E * dt.abs())
    assert status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_cross_entropy_rows_do_not_depend_on_the_batch(dtype):
    M, D, V = 700, 136, 9000
    x, table, t = xent_case(M, D, V, dtype, 5, kept=0.9)
    loss, lse = cg.linear_cross_entropy_fwd(x, table, t, reduction="none")
    dx, _ = cg.linear_cross_entropy_bwd(torch.ones(M, device="cuda"), x, table, t, lse, reduction="none")
    for a, b in ((0, 1), (13, 14), (100, 229), (699, 700), (0, 513)):
        part = [v[a:b].contiguous() for v in (x, t, lse)]
        l2, lse2 = cg.linear_cross_entropy_fwd(part[0], table, part[1], reduction="none")
        assert same_bits(l2, loss[a:b]) and same_bits(lse2, lse[a:b])
        d2, _ = cg.linear_cross_entropy_bwd(torch.ones(b - a, device="cuda"), part[0], table, part[1], lse2,
                                            reduction="none")
        assert same_bits(d2, dx[a:b])


def test_cross_entropy_large_batch_matches_small_ones():
    """Enough positions that the vocabulary goes in pieces and dx's granules
    are added in place: the rows agree bit for bit with small calls, whose
    granules lie side by side."""
    M, D, V = 9000, 64, 13000
    x, table, t = xent_case(M, D, V, "bf16", 6, kept=1.0)
    loss, lse = cg.linear_cross_entropy_fwd(x, table, t, reduction="none")
    g = torch.ones(M, device="cuda")
    dx, dt = cg.linear_cross_entropy_bwd(g, x, table, t, lse, reduction="none")
    for a, b in ((0, 100), (4090, 4500), (8999, 9000)):
        sl = slice(a, b)
        l2, _ = cg.linear_cross_entropy_fwd(x[sl], table, t[sl], reduction="none")
        d2, _ = cg.linear_cross_entropy_bwd(g[sl], x[sl], table, t[sl], lse[sl], reduction="none")
        assert same_bits(l2, loss[sl]) and same_bits(d2, dx[sl])
    _, _, _, _, wdx, wdt, edx, edt = xent_reference(x, table, t, g)
    within(dx, wdx, edx)
    within(dt, wdt, edt)
    again = cg.linear_cross_entropy_bwd(g, x, table, t, lse, reduction="none")
    assert same_bits(again[0], dx) and same_bits(again[1], dt)


@pytest.mark.parametrize("reduction", ["none", "mean"])
def test_cross_entropy_long_list(reduction):
    """More positions than a tile kernel's preparation counts by itself."""
    M, D, V = 20011, 64, 300
    x, table, t = xent_case(M, D, V, "bf16", 21, kept=0.6)
    grad = torch.randn(M, generator=gen(22), device="cuda") if reduction == "none" else torch.tensor(2.0, device="cuda")
    count = int((t >= 0).sum())
    rows = grad if reduction == "none" else torch.full((M,), 2.0 / count, device="cuda", dtype=torch.float64)
    loss, lse, keep, eloss, dx, dt, edx, edt = xent_reference(x, table, t, rows)
    got, glse = cg.linear_cross_entropy_fwd(x, table, t, reduction=reduction)
    within(glse, torch.where(keep, lse, 0.0), eloss)
    if reduction == "none":
        within(got, loss, eloss)
    else:
        within(got, loss.sum() / count, eloss.sum() / count)
    gdx, gdt = cg.linear_cross_entropy_bwd(grad, x, table, t, glse, reduction=reduction)
    within(gdx, dx, edx + 2 * E * dx.abs())
    within(gdt, dt, edt + 2 * E * dt.abs())
    assert not bool(gdx[~keep].any()) and status() == 0


def test_cross_entropy_ignored_positions_hold_anything():
    M, D, V = 300, 64, 500
    x, table, t = xent_case(M, D, V, "bf16", 8, kept=0.5)
    bad = x.clone()
    bad[t == -100] = float("nan")
    bad[(t == -100).nonzero()[0]] = float("inf")
    one = torch.tensor(1.0, device="cuda")
    ref = cg.linear_cross_entropy_fwd(x, table, t)
    got = cg.linear_cross_entropy_fwd(bad, table, t)
    assert same_bits(ref[0], got[0]) and same_bits(ref[1], got[1])
    a, b = (cg.linear_cross_entropy_bwd(one, v, table, t, ref[1]) for v in (x, bad))
    assert same_bits(a[0], b[0]) and same_bits(a[1], b[1])
    # another index to ignore
    t2 = torch.where(t == -100, 3, t)
    got = cg.linear_cross_entropy_fwd(x, table, t2, ignore_index=3)
    keep = t2 != 3
    want, _ = cg.linear_cross_entropy_fwd(x[keep], table, t2[keep])
    within(got[0], want.double(), 4 * E * want.double().abs())


@pytest.mark.parametrize("M", [1, 257])
def test_cross_entropy_without_positions_that_count(M):
    D, V = 64, 300
    x, table, _ = xent_case(M, D, V, "f16", 9)
    t = torch.full((M,), -100, device="cuda")
    for red in ("mean", "sum"):
        loss, lse = cg.linear_cross_entropy_fwd(x, table, t, reduction=red)
        assert float(loss) == 0.0 and not bool(lse.any())
        dx, dt = cg.linear_cross_entropy_bwd(torch.tensor(1.0, device="cuda"), x, table, t, lse, reduction=red)
        assert not bool(dx.any()) and not bool(dt.any())
    loss, lse = cg.linear_cross_entropy_fwd(x, table, t, reduction="none")
    dx, dt = cg.linear_cross_entropy_bwd(torch.ones(M, device="cuda"), x, table, t, lse, reduction="none")
    assert not bool(loss.any()) and not bool(dx.any()) and not bool(dt.any())
    # and no positions at all
    e = torch.empty(0, D, dtype=torch.float16, device="cuda")
    te = torch.empty(0, dtype=torch.int64, device="cuda")
    loss, lse = cg.linear_cross_entropy_fwd(e, table, te)
    assert float(loss) == 0.0
    dx, dt = cg.linear_cross_entropy_bwd(torch.tensor(1.0, device="cuda"), e, table, te, lse)
    assert dx.shape == (0, D) and not bool(dt.any())
    assert status() == 0


def test_cross_entropy_targets_outside_the_table():
    x, table, t = xent_case(40, 64, 100, "bf16", 10, kept=1.0)
    wrong = t.clone()
    wrong[3], wrong[7], wrong[30] = 100, -1, 2 ** 40
    loss, lse = cg.linear_cross_entropy_fwd(x, table, wrong)
    assert status() == 7 and status() == 0
    out = t.clone()
    out[[3, 7, 30]] = -100
    ref, ref_lse = cg.linear_cross_entropy_fwd(x, table, out)
    assert same_bits(loss, ref) and same_bits(lse, ref_lse)
    one = torch.tensor(1.0, device="cuda")
    a = cg.linear_cross_entropy_bwd(one, x, table, wrong, lse)
    assert status() == 7
    b = cg.linear_cross_entropy_bwd(one, x, table, out, lse)
    assert same_bits(a[0], b[0]) and same_bits(a[1], b[1])


def test_cross_entropy_large_logits():
    """Logits of hundreds: no overflow, probabilities of exactly 0 and 1."""
    M, D, V = 65, 64, 1000
    x, table, t = xent_case(M, D, V, "bf16", 12, kept=1.0)
    x = x * 64
    g = torch.ones(M, device="cuda")
    loss, lse, keep, eloss, dx, dt, edx, edt = xent_reference(x, table, t, g)
    got, glse = cg.linear_cross_entropy_fwd(x, table, t, reduction="none")
    within(got, loss, eloss)
    gdx, gdt = cg.linear_cross_entropy_bwd(g, x, table, t, glse, reduction="none")
    within(gdx, dx, edx)
    within(gdt, dt, edt)


def test_cross_entropy_gradient_against_differences():
    M, D, V = 33, 64, 300
    x, table, t = xent_case(M, D, V, "f16", 13)
    g = gen(14)
    d = torch.randn(M, D, generator=g, device="cuda", dtype=torch.float64)
    dw = torch.randn(V, D, generator=g, device="cuda", dtype=torch.float64)
    keep = t >= 0

    def f(X, W):
        z = X @ W.t()
        return (torch.logsumexp(z, 1) - z.gather(1, t.clamp(min=0)[:, None])[:, 0])[keep].sum()

    h = 1e-4
    X, W = x.double(), table.double()
    num = (f(X + h * d, W + h * dw) - f(X - h * d, W - h * dw)) / (2 * h)
    _, lse = cg.linear_cross_entropy_fwd(x, table, t, reduction="sum")
    dx, dt = cg.linear_cross_entropy_bwd(torch.tensor(1.0, device="cuda"), x, table, t, lse, reduction="sum")
    edx, edt = xent_reference(x, table, t, torch.ones(M, device="cuda"))[6:]
    got = (dx.double() * d).sum() + (dt.double() * dw).sum()
    lim = ((edx + U[x.dtype] * dx.double().abs()) * d.abs()).sum() + ((edt + U[x.dtype] * dt.double().abs()) * dw.abs()).sum()
    assert abs(float(num - got)) <= float(lim) + 1e-3


# ---- streams, autograd, the operators together ---------------------------------------------

def test_calls_on_another_stream():
    """Workspaces belong to the call's stream: calls in flight on two streams,
    allocations in between, same results."""
    x, table, t = xent_case(600, 256, 6000, "bf16", 15)
    ids = t.clamp(min=0)
    ref = cg.linear_cross_entropy_fwd(x, table, t)
    one = torch.tensor(1.0, device="cuda")
    ref_bwd = cg.linear_cross_entropy_bwd(one, x, table, t, ref[1])
    ref_emb = cg.embedding_bwd(x, ids, 6000)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        outs = []
        for s in streams:
            for handle in (s, s.cuda_stream):
                loss, lse = cg.linear_cross_entropy_fwd(x, table, t, stream=handle)
                bwd = cg.linear_cross_entropy_bwd(one, x, table, t, lse, stream=handle)
                emb = cg.embedding_bwd(x, ids, 6000, stream=handle)
                outs.append((loss, lse, *bwd, emb))
            junk = [torch.full((1 << 20,), 7.0, device="cuda") for _ in range(4)]
        torch.cuda.synchronize()
        del junk
        for o in outs:
            assert all(same_bits(a, b) for a, b in zip(o, (*ref, *ref_bwd, ref_emb)))


def test_refusals():
    x, table, t = xent_case(16, 64, 100, "bf16", 16)
    with pytest.raises(ValueError):
        cg.linear_cross_entropy_fwd(x.t().contiguous().t(), table, t)       # not contiguous
    with pytest.raises(TypeError):
        cg.linear_cross_entropy_fwd(x, table, t.int())
    with pytest.raises(TypeError):
        cg.linear_cross_entropy_fwd(x, table.half(), t)
    with pytest.raises(cg.CarbonError) as e:
        cg.linear_cross_entropy_fwd(x.float(), table.float(), t)
    assert e.value.status == 2
    with pytest.raises(cg.CarbonError) as e:
        cg.linear_cross_entropy_fwd(x[:, :60].contiguous(), table[:, :60].contiguous(), t)
    assert e.value.status == 3
    with pytest.raises(ValueError):
        cg.linear_cross_entropy_fwd(x, table, t[:-1])
    with pytest.raises(ValueError):
        cg.rms_norm_bwd(x, table[0], torch.ones(16, device="cuda"))
    with pytest.raises(TypeError):
        cg.embedding_fwd(table, t.int())
    with pytest.raises(ValueError):
        cg.embedding_bwd(x, t, 100, accumulate_to=torch.zeros(99, 64, dtype=x.dtype, device="cuda"))
    with pytest.raises(cg.CarbonError) as e:
        cg.embedding_bwd(x, t, 100, padding_idx=100)
    assert e.value.status == 1


@pytest.mark.parametrize("tier", ["exact", "tc"])
def test_norm_linear_is_norm_then_linear(tier):
    """Forward: the same bits as the two layers.  Backward: dX from the same
    product; the checkpoint's values stand for the normalised rows."""
    g, dt = gen(17), torch.bfloat16
    M, D, N = 96, 64, 72
    x, res = randn(g, 2, M // 2, D, dtype=dt), randn(g, 2, M // 2, D, dtype=dt)
    gamma, w, b = randn(g, D, dtype=dt), randn(g, D, N, dtype=dt, std=0.1), randn(g, N, dtype=dt)
    leaves = [v.clone().requires_grad_(True) for v in (x, res, gamma, w, b)]
    out, h = cnn.norm_linear(leaves[0], leaves[2], leaves[3], leaves[4], residual=leaves[1], tier=tier)
    y2, h2 = cnn.rms_norm(x, gamma, res)
    assert same_bits(out.detach(), cnn.deterministic_linear(y2, w, b, tier)) and same_bits(h.detach(), h2)
    dout, dh = randn(g, 2, M // 2, N, dtype=dt), randn(g, 2, M // 2, D, dtype=dt)
    torch.autograd.backward([out, h], [dout, dh])
    r = cg.rms_norm_fwd(x.view(M, D), gamma, res.view(M, D), quantize=True)
    dy = cg.linear_dx(dout.view(M, N), w, tier=tier)
    dx, dgamma, y = cg.rms_norm_bwd(dy, gamma, r.rstd, codes=r.codes, scales=r.scales, dh=dh.view(M, D), recompute=True)
    assert same_bits(leaves[0].grad.view(M, D), dx) and same_bits(leaves[1].grad.view(M, D), dx)
    assert same_bits(leaves[2].grad, dgamma)
    assert same_bits(leaves[3].grad, cg.linear_dw(y, dout.view(M, N), tier=tier))
    assert same_bits(leaves[4].grad, cnn.bias_grad(dout.view(M, N)))


def test_modules_and_tied_weights():
    V, D, M = 300, 64, 50
    g = gen(18)
    torch.manual_seed(3)
    emb = cnn.Embedding(V, D, scale=2.0, padding_idx=4, device="cuda", dtype=torch.bfloat16)
    norm = cnn.RMSNorm(D, device="cuda", dtype=torch.bfloat16)
    ids = torch.randint(0, V, (5, M // 5), generator=g, device="cuda")
    t = torch.randint(0, V, (5, M // 5), generator=g, device="cuda")
    y = norm(emb(ids))
    loss = cnn.linear_cross_entropy(y, emb.weight, t)
    loss.backward()
    # the table's gradient: the output layer's plus the lookup's
    yv = y.detach().view(M, D)
    l2, lse = cg.linear_cross_entropy_fwd(yv, emb.weight.detach(), t.view(-1))
    assert same_bits(loss.detach(), l2)
    dx, dt = cg.linear_cross_entropy_bwd(torch.tensor(1.0, device="cuda"), yv, emb.weight.detach(), t.view(-1), lse)
    e = cg.embedding_fwd(emb.weight.detach(), ids, 2.0).view(M, D)
    r = cg.rms_norm_fwd(e, norm.weight.detach())
    de, dgamma = cg.rms_norm_bwd(dx, norm.weight.detach(), r.rstd, h=e)
    assert same_bits(norm.weight.grad, dgamma)
    want = dt.double() + cg.embedding_bwd(de, ids.view(-1), V, 2.0, padding_idx=4).double()
    # autograd rounds the lookup's gradient before it adds the two
    assert bool(((emb.weight.grad.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -133).all())
    acc = dt.clone()
    cg.embedding_bwd(de, ids.view(-1), V, 2.0, padding_idx=4, accumulate_to=acc)
    assert bool(((acc.double() - want).abs() <= 2.0 ** -7 * (want.abs() + dt.double().abs())).all())


def test_training_example_repeats_bit_for_bit():
    from examples import train_tied_lm as ex
    a = ex.train(1000, 64, 2, 300, 12)
    b = ex.train(1000, 64, 2, 300, 12)
    assert a == b
    assert a[0][-1] < a[0][0]
    assert status() == 0
