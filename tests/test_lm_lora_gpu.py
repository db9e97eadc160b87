"""The linear layer with low-rank adapters and its gradients, against float64."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import deterministic_invariant_gemm_fwd_gb300 as cg  # noqa: E402
from deterministic_invariant_gemm_fwd_gb300 import nn  # noqa: E402
from tests.test_lm_gpu import U, gen, same_bits, status  # noqa: E402

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
# what the pair of 16-bit terms leaves of u, relative; the output's half steps near zero
TERMS = {torch.bfloat16: 2.0 ** -17, torch.float16: 2.0 ** -22}
STEP = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}


class Case:
    def __init__(self, M, K, N, n, r, dtype, seed, mix="runs", bias=True, size=1.0):
        g = gen(seed)
        dt = DT[dtype]

        def make(*shape, std=1.0):
            return (torch.randn(*shape, generator=g, device="cuda") * std).to(dt)
        self.x, self.dy = make(M, K), make(M, N, std=size)
        self.w = make(K, N, std=1 / math.sqrt(K))
        self.bias = make(N) if bias else None
        self.a, self.b = make(n, K, r, std=1 / math.sqrt(K)), make(n, r, N, std=1 / math.sqrt(r))
        self.scales = torch.rand(n, generator=g, device="cuda") * 2 - 0.5
        if mix == "one":
            ids = torch.zeros(M, dtype=torch.long, device="cuda")
        elif mix == "any":
            ids = torch.randint(-1, n, (M,), generator=g, device="cuda")
        else:                                               # runs of rows
            run = torch.cumsum((torch.rand(M, generator=g, device="cuda") < 0.02).long(), 0)
            ids = torch.randint(-1, n, (M + 1,), generator=g, device="cuda")[run]
        self.ids = ids

    def fwd(self):
        return cg.lora_linear_fwd(self.x, self.w, self.a, self.b, self.ids, self.scales, self.bias, keep=True)

    def bwd(self, u, **kw):
        return cg.lora_linear_bwd(self.dy, self.x, self.w, self.a, self.b, self.ids, self.scales, u, **kw)


def near(got, want, bound, dtype):
    """bound: of the value before it is rounded."""
    lim = bound * (1 + U[dtype]) + U[dtype] * want.abs() + STEP[dtype]
    assert bool(((got.double() - want).abs() <= lim).all()), float(((got.double() - want).abs() / lim).max())


def check(c, again=True):
    """Forward and gradients.  eu: of u, a sum of K products in an accumulator
    that may truncate, the scale, the addition of up to eight pieces; the terms
    leave TERMS of it and fp16's step."""
    dt = c.x.dtype
    y, u = c.fwd()
    dx, da, db = c.bwd(u)
    assert status() == 0
    X, W, A, B, dY = (t.double() for t in (c.x, c.w, c.a, c.b, c.dy))
    M, K = X.shape
    N, n, r = W.shape[1], A.shape[0], A.shape[2]
    acc = 2.0 ** -23
    Y, eY = X @ W, (K + 2 * r + 2) * acc * (X.abs() @ W.abs())
    if c.bias is not None:
        Y, eY = Y + c.bias.double(), eY + acc * c.bias.double().abs()
    dX, edX = dY @ W.t(), (N + 2 * r + 2) * acc * (dY.abs() @ W.abs().t())
    dA, dB, edA, edB = (torch.zeros(s.shape, dtype=torch.float64, device="cuda") for s in (A, B, A, B))
    step = 2.0 ** -25 if dt == torch.float16 else 0.0
    for i in range(n):
        at = (c.ids == i).nonzero()[:, 0]
        s = float(c.scales[i].double())
        x, dy = X[at], dY[at]
        uu, eu = s * (x @ A[i]), abs(s) * (K + 12) * acc * (x.abs() @ A[i].abs())
        du, edu = s * (dy @ B[i].t()), abs(s) * (N + 12) * acc * (dy.abs() @ B[i].abs().t())
        tu, tdu = eu + TERMS[dt] * (uu.abs() + eu), edu + TERMS[dt] * (du.abs() + edu)
        Y[at] += uu @ B[i]
        eY[at] += (tu + step) @ B[i].abs() + (K + 2 * r + 2) * acc * ((uu.abs() + tu) @ B[i].abs())
        dX[at] += du @ A[i].t()
        edX[at] += (tdu + step) @ A[i].abs().t() + (N + 2 * r + 2) * acc * ((du.abs() + tdu) @ A[i].abs().t())
        # the third term has 11 more bits below fp16's step
        rows = at.numel() + 4
        dA[i], dB[i] = x.t() @ du, uu.t() @ dy
        edA[i] = x.abs().t() @ (tdu + step * 2.0 ** -11) + rows * acc * (x.abs().t() @ (du.abs() + tdu))
        edB[i] = (tu + step * 2.0 ** -11).t() @ dy.abs() + rows * acc * ((uu.abs() + tu).t() @ dy.abs())
    for got, want, bound in ((y, Y, eY), (dx, dX, edX), (da, dA, edA), (db, dB, edB)):
        assert got.shape == want.shape and got.dtype == dt
        near(got, want, bound, dt)
    if again:
        y2, u2 = c.fwd()
        assert same_bits(y2, y) and same_bits(u2, u)
        assert all(same_bits(p, q) for p, q in zip(c.bwd(u), (dx, da, db)))
    return y, u, dx, da, db


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("mix", ["one", "runs", "any"])
@pytest.mark.parametrize("M,K,N,n,r", [
    (1, 8, 8, 1, 8), (1, 768, 768, 4, 16), (3, 64, 72, 2, 24), (64, 768, 2304, 24, 16), (130, 136, 264, 5, 32),
    (255, 520, 776, 3, 64), (257, 320, 200, 7, 40), (511, 1096, 136, 2, 128), (513, 72, 1032, 300, 8),
    (1500, 264, 328, 3, 72), (3001, 520, 776, 9, 104),
])
def test_layer_and_gradients(M, K, N, n, r, dtype, mix):
    check(Case(M, K, N, n, r, dtype, M + K + N + r, mix, bias=M % 2 == 0))


@pytest.mark.parametrize("mix", ["one", "runs"])
def test_many_tiles(mix):
    check(Case(8192, 768, 2304, 4, 16, "bf16", 1, mix))
    check(Case(2049, 2048, 4096, 4, 16, "f16", 2, mix), again=False)


def test_a_row_does_not_depend_on_the_others():
    c = Case(1100, 264, 520, 6, 24, "bf16", 3, "any")
    y, u, dx, _, _ = check(c, again=False)
    for a, b in ((0, 1), (7, 300), (600, 1100)):
        p = Case(1, 264, 520, 6, 24, "bf16", 3)
        p.__dict__.update({k: v for k, v in c.__dict__.items()})
        p.x, p.dy, p.ids = c.x[a:b].contiguous(), c.dy[a:b].contiguous(), c.ids[a:b].contiguous()
        py, pu = p.fwd()
        pdx, _, _ = p.bwd(pu)
        assert same_bits(py, y[a:b]) and same_bits(pu, u[a:b]) and same_bits(pdx, dx[a:b])
    # an adapter's gradients come from its own rows alone, in their order
    mine = (c.ids == 2).nonzero()[:, 0]
    p.x, p.dy, p.ids = c.x[mine].contiguous(), c.dy[mine].contiguous(), c.ids[mine].contiguous()
    _, da, db = c.bwd(u)
    _, pda, pdb = p.bwd(p.fwd()[1])
    assert same_bits(pda[2], da[2]) and same_bits(pdb[2], db[2])
    others = torch.arange(6, device="cuda") != 2
    assert bool((pda[others] == 0).all()) and bool((pdb[others] == 0).all())


def test_rows_without_an_adapter():
    c = Case(300, 136, 264, 3, 16, "bf16", 4, "any")
    y, _ = c.fwd()
    plain = cg.linear_fwd(c.x, c.w, c.bias, tier="tc")
    bare = c.ids < 0
    assert same_bits(y[bare], plain[bare])
    c.ids[:] = -1
    y, u = c.fwd()
    dx, da, db = c.bwd(u)
    assert same_bits(y, plain) and same_bits(dx, cg.linear_dx(c.dy, c.w, tier="tc"))
    assert bool((da == 0).all()) and bool((db == 0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_nothing_of_other_rows_or_adapters_reaches_a_row(dtype):
    c = Case(700, 136, 264, 4, 16, dtype, 5, "any")
    y, u = c.fwd()
    dx, da, db = c.bwd(u)
    bad = Case(700, 136, 264, 4, 16, dtype, 5, "any")
    for t, k in ((bad.a, 1), (bad.b, 1)):                    # an adapter of NaN and infinities
        t[k] = math.nan
        t[k, 0] = math.inf
    bad.scales[1] = math.nan
    bad.x[bad.ids == -1] = math.nan                          # rows that hold nothing
    bad.dy[bad.ids == -1] = math.inf
    ok = (c.ids != 1) & (c.ids != -1)
    y2, u2 = bad.fwd()
    dx2, da2, db2 = bad.bwd(u2)
    assert same_bits(y2[ok], y[ok]) and same_bits(dx2[ok], dx[ok])
    keep = torch.tensor([0, 2, 3], device="cuda")
    assert same_bits(da2[keep], da[keep]) and same_bits(db2[keep], db[keep])
    assert bool(y2[c.ids == 1].isnan().all())


def test_numbers_that_name_no_adapter():
    c = Case(200, 64, 64, 3, 8, "bf16", 6, "any")
    ref, _ = c.fwd()
    assert status() == 0
    c.ids[5], c.ids[150] = 3, -7
    y, u = c.fwd()
    assert cg.carbon_get_device_status() == 7
    rest = torch.ones(200, dtype=torch.bool, device="cuda")
    rest[5] = rest[150] = False
    plain = cg.linear_fwd(c.x, c.w, c.bias, tier="tc")
    assert same_bits(y[rest], ref[rest]) and same_bits(y[~rest], plain[~rest])
    c.bwd(u)
    assert cg.carbon_get_device_status() == 7
    assert status() == 0


@pytest.mark.parametrize("size", [1e-7, 1e-5, 100.0])
def test_small_and_large_gradients_in_fp16(size):
    check(Case(900, 136, 264, 3, 16, "f16", 7, "runs", size=size))


def test_no_rows():
    c = Case(8, 64, 72, 3, 8, "bf16", 8)
    c.x, c.dy, c.ids = c.x[:0], c.dy[:0], c.ids[:0]
    y, u = c.fwd()
    dx, da, db = c.bwd(u)
    assert y.shape == (0, 72) and dx.shape == (0, 64) and bool((da == 0).all()) and bool((db == 0).all())


def test_parts_of_the_gradient():
    c = Case(700, 136, 264, 4, 16, "bf16", 9)
    _, u = c.fwd()
    dx, da, db = c.bwd(u)
    only = c.bwd(u, need_adapters=False)
    assert same_bits(only[0], dx) and only[1] is None and only[2] is None
    only = c.bwd(u, need_dx=False)
    assert only[0] is None and same_bits(only[1], da) and same_bits(only[2], db)
    assert c.bwd(u, need_dx=False, need_adapters=False) == (None, None, None)


def test_gradient_against_differences():
    c = Case(70, 64, 72, 3, 8, "f16", 10, "any", bias=False)
    g = gen(11)
    dirs = [torch.randn(t.shape, generator=g, device="cuda", dtype=torch.float64) for t in (c.x, c.a, c.b)]
    at, live = c.ids.clamp(min=0), (c.ids >= 0).double() * c.scales.double()[c.ids.clamp(min=0)]

    def f(X, A, B):
        u = torch.einsum("mk,mkr->mr", X, A[at]) * live[:, None]
        return ((X @ c.w.double() + torch.einsum("mr,mrn->mn", u, B[at])) * c.dy.double()).sum()

    h = 1e-4
    at0 = [t.double() for t in (c.x, c.a, c.b)]
    num = (f(*(t + h * d for t, d in zip(at0, dirs))) - f(*(t - h * d for t, d in zip(at0, dirs)))) / (2 * h)
    got = c.bwd(c.fwd()[1])
    total = sum((p.double() * d).sum() for p, d in zip(got, dirs))
    mag = sum((p.double().abs() * d.abs()).sum() for p, d in zip(got, dirs))
    # each result is off by half a step of fp16 and as little again from fp32 sums; the differences by h^2
    assert abs(float(num - total)) <= 2 * U[torch.float16] * float(mag) + 1e-2


def test_another_stream_and_a_graph():
    c = Case(700, 264, 520, 5, 16, "bf16", 12)
    y, u = c.fwd()
    ref = (y, *c.bwd(u))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y2, u2 = cg.lora_linear_fwd(c.x, c.w, c.a, c.b, c.ids, c.scales, c.bias, keep=True, stream=side)
    y3, _ = c.fwd()
    back = c.bwd(u2, stream=side)
    torch.cuda.synchronize()
    assert all(same_bits(p, q) for p, q in zip((y2, *back), ref)) and same_bits(y3, y)
    ids = torch.full_like(c.ids, -1)
    keep, c.ids = c.ids, ids
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y4, u4 = c.fwd()
        back = c.bwd(u4)
    ids.copy_(keep)                                          # the replay's adapters
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert all(same_bits(p, q) for p, q in zip((y4, *back), ref))


def test_autograd_and_module():
    torch.manual_seed(0)
    base = nn.Linear(136, 264, tier="tc", device="cuda", dtype=torch.bfloat16)
    layer = nn.LoraLinear(base, adapters=3, rank=8, alpha=16)
    x = torch.randn(4, 50, 136, device="cuda").bfloat16().requires_grad_()
    ids = torch.randint(-1, 3, (4, 50), device="cuda")
    assert same_bits(layer(x, ids), base(x))                 # b is zero
    with torch.no_grad():
        layer.b.normal_(std=0.1)
    y = layer(x, ids)
    dy = torch.randn_like(y)
    y.backward(dy)
    assert layer.weight.grad is None and layer.bias.grad is None
    x2 = x.detach().view(200, 136)
    _, u = cg.lora_linear_fwd(x2, layer.weight, layer.a.detach(), layer.b.detach(), ids.view(-1), layer.scales, layer.bias, keep=True)
    dx, da, db = cg.lora_linear_bwd(dy.view(200, 264), x2, layer.weight, layer.a.detach(), layer.b.detach(), ids.view(-1),
                                    layer.scales, u)
    assert same_bits(x.grad.view(200, 136), dx) and same_bits(layer.a.grad, da) and same_bits(layer.b.grad, db)
    one = layer(x, 2)
    assert same_bits(one, layer(x, torch.full_like(ids, 2)))
    full = nn.LoraLinear(nn.Linear(136, 264, tier="tc", device="cuda", dtype=torch.bfloat16), 2, 8, train_base=True)
    full(x, 0).sum().backward()
    assert full.weight.grad.shape == (136, 264) and full.bias.grad.shape == (264,)
    with pytest.raises(ValueError):
        layer(x, ids.view(-1))
    with pytest.raises(ValueError, match="scales"):
        nn.lora_linear(x, layer.weight, layer.a, layer.b, ids, layer.scales.clone().requires_grad_())
    layer.bfloat16()                                         # casts the scales as well
    assert same_bits(layer(x, ids), y)
    (gx,) = torch.autograd.grad(layer(x, ids).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="no derivative"):
        gx.sum().backward()


def test_first_call_of_a_thread():
    """Tensor maps are encoded in a thread that has made no CUDA call yet."""
    import threading
    c = Case(64, 64, 72, 2, 8, "bf16", 13)
    y, u = c.fwd()
    ref = c.bwd(u)
    dx = cg.linear_dx(c.dy, c.w, tier="tc")
    for call, want in ((lambda: c.bwd(u), ref), (lambda: (cg.linear_dx(c.dy, c.w, tier="tc"),), (dx,))):
        got = []
        t = threading.Thread(target=lambda: got.append(call()))
        t.start()
        t.join()
        assert got and all(same_bits(p, q) for p, q in zip(got[0], want))
