"""The norm of all gradients and their clipping, against float64."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import deterministic_invariant_gemm_fwd_gb300 as cg  # noqa: E402
from deterministic_invariant_gemm_fwd_gb300 import nn  # noqa: E402

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
BLOCK = 2048                            # elements that a warp takes at a time
# Relative errors in units of 2^-24.  The norm: a chain of 16 fused additions and
# two more, halved by the square root, and its own rounding.  The factor: the
# norm's, an addition and a division.
NORM, FACTOR = 10, 12
TINY = {F32: 2.0 ** -150, BF16: 2.0 ** -134, F16: 2.0 ** -25}      # half the smallest step


def make(sizes, types, std=1.0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(n, generator=g, device="cuda") * std).to(types[i % len(types)]) for i, n in enumerate(sizes)]


def check(grads, max_norm, out, norm, eps=1e-6):
    want = math.sqrt(sum(float((t.double() ** 2).sum()) for t in grads))
    assert abs(float(norm) - want) <= NORM * 2.0 ** -24 * want
    factor = min(1.0, max_norm / (want + eps))
    for t, o in zip(grads, out):
        assert o.dtype == t.dtype and o.shape == t.shape
        exact = t.double() * factor
        bound = exact.abs() * ((FACTOR + 1) * 2.0 ** -24 + torch.finfo(t.dtype).eps / 2) * 1.001 + TINY[t.dtype]
        assert bool(((o.double() - exact).abs() <= bound).all())


@pytest.mark.parametrize("types", [[F32], [BF16], [F16], [BF16, F32, F16]], ids=["f32", "bf16", "f16", "mixed"])
@pytest.mark.parametrize("sizes", [
    [1], [7, 0, 9], [BLOCK], [BLOCK - 1, BLOCK + 1], [3 * BLOCK + 5, 1, 2, 3], [257] * 300, [0, 0], [1000003],
    [3] * 32, [3] * 33, [0] * 300 + [5], [2 * BLOCK + 1] * 257,
], ids=str)
def test_norm_and_clipping(sizes, types):
    grads = make(sizes, types)
    for max_norm in (0.5, 1e9):
        out = [torch.full_like(t, 7.0) for t in grads]
        norm = cg.clip_grads(grads, max_norm, out=out)
        check(grads, max_norm, out, norm)
        assert torch.equal(cg.grad_norm(grads), norm)
        mine = [t.clone() for t in grads]
        assert torch.equal(cg.clip_grads(mine, max_norm), norm)
        assert all(torch.equal(a, b) for a, b in zip(mine, out))
    assert cg.carbon_get_device_status() == 0


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_addresses_do_not_matter(dtype):
    """Tensors that start between 16-byte boundaries: the same bits."""
    base = make([2 * BLOCK + 77, 5003, 1], [dtype])
    want = [torch.empty_like(t) for t in base]
    norm = cg.clip_grads(base, 1.0, out=want)
    for shift in range(1, 8):
        moved = [torch.cat([t.new_zeros(shift), t])[shift:] for t in base]
        out = [torch.empty(t.numel() + 9, dtype=dtype, device="cuda").fill_(3.0) for t in base]
        views = [o[3:3 + t.numel()] for o, t in zip(out, base)]
        assert torch.equal(cg.clip_grads(moved, 1.0, out=views), norm)
        for o, v, w in zip(out, views, want):
            assert torch.equal(v, w)
            assert bool((o[:3] == 3.0).all()) and bool((o[3 + w.numel():] == 3.0).all())     # nothing beside it


def test_several_chunks_per_warp():
    """More chunks than warps, and runs of them that end inside a tensor."""
    grads = make([5000 * BLOCK + 3, 5, 7 * BLOCK + 9], [BF16, F32, F16], std=1e-3)
    out = [torch.empty_like(t) for t in grads]
    check(grads, 0.25, out, cg.clip_grads(grads, 0.25, out=out))


@pytest.mark.parametrize("dtype,size", [(F32, 1e-30), (F32, 1e-44), (F32, 1e30), (F32, 3e38 / 256), (BF16, 1e-38),
                                        (BF16, 1e36), (F16, 1e-7), (F16, 6e4)])
def test_squares_outside_fp32(dtype, size):
    """Norms that are fp32 numbers although the squares are none; values are
    multiples of one size so that the type's rounding of them does not matter."""
    g = torch.Generator(device="cuda").manual_seed(3)
    one = torch.tensor(size, device="cuda").to(dtype)
    t = torch.where(torch.rand(20000, generator=g, device="cuda") < 0.5, one, -one)
    want = float(one.double().abs()) * math.sqrt(20000.0)
    assert abs(float(cg.grad_norm([t])) - want) <= NORM * 2.0 ** -24 * want + 2.0 ** -150
    mixed = [t, torch.zeros(5, device="cuda"), torch.zeros(70000, device="cuda", dtype=BF16)]
    assert torch.equal(cg.grad_norm(mixed), cg.grad_norm([t]))


def test_nan_infinity_and_zero():
    for bad in (math.nan, math.inf, -math.inf):
        t = [torch.ones(100, device="cuda"), torch.ones(100, device="cuda", dtype=BF16)]
        t[1][3] = bad
        norm = cg.clip_grads(t, 1.0)
        if math.isnan(bad):
            assert math.isnan(float(norm)) and bool(t[0].isnan().all()) and bool(t[1].isnan().all())
        else:
            assert math.isinf(float(norm)) and bool((t[0] == 0).all()) and bool(t[1][3].isnan())
    z = [torch.zeros(9, device="cuda")]
    assert float(cg.clip_grads(z, 1.0)) == 0.0 and bool((z[0] == 0).all())
    assert float(cg.clip_grads([], 1.0)) == 0.0
    small = make([1000], [BF16], std=1e-3)
    before = small[0].clone()
    cg.clip_grads(small, 5.0)
    assert torch.equal(small[0], before)                     # the factor is 1


def test_other_stream_and_graph():
    grads = make([4097, 33], [BF16, F32])
    want = [torch.empty_like(t) for t in grads]
    norm = cg.clip_grads(grads, 1.0, out=want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out = [torch.empty_like(t) for t in grads]
    side.wait_stream(torch.cuda.current_stream())
    n2 = cg.clip_grads(grads, 1.0, out=out, stream=side)
    side.synchronize()
    assert torch.equal(n2, norm) and all(torch.equal(a, b) for a, b in zip(out, want))
    mine = [t.clone() for t in grads]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        n3 = cg.clip_grads(mine, 1.0)
    for _ in range(2):                                        # a replay reads what the tensors hold then
        for a, b in zip(mine, grads):
            a.copy_(b)
        graph.replay()
        assert torch.equal(n3, norm) and all(torch.equal(a, b) for a, b in zip(mine, want))


def test_parameters():
    p = [torch.nn.Parameter(torch.zeros(5, 3, device="cuda")), torch.nn.Parameter(torch.zeros(4, device="cuda")),
         torch.nn.Parameter(torch.zeros(2, device="cuda"))]
    p[0].grad, p[1].grad = torch.full((5, 3), 2.0, device="cuda"), torch.full((4,), -1.0, device="cuda")
    norm = nn.clip_grad_norm_(p, 1.0)
    assert abs(float(norm) - 8.0) <= 8 * 2.0 ** -20 and abs(float(p[0].grad[0, 0]) - 0.25) <= 2.0 ** -20
    assert p[2].grad is None
    assert float(nn.clip_grad_norm_(p[2], 1.0)) == 0.0


def test_refusals_on_a_gpu():
    t = torch.ones(64, device="cuda")
    with pytest.raises(cg.CarbonError, match="INVALID_ARG"):
        cg.clip_grads([t, t], 1.0)                            # scaled twice at once
    with pytest.raises(cg.CarbonError, match="INVALID_ARG"):
        cg.clip_grads([t[:40], t[39:]], 1.0)
    with pytest.raises(cg.CarbonError, match="INVALID_ARG"):
        cg.clip_grads([t[:32]], 1.0, out=[t[31:63]])
    with pytest.raises(ValueError):
        cg.clip_grads([torch.ones(4, 6, device="cuda").t()], 1.0)
    with pytest.raises(ValueError):
        cg.clip_grads([t], -1.0)
    with pytest.raises(ValueError):
        cg.clip_grads([t], 1.0, out=[t[:5]])
    with pytest.raises(TypeError):
        cg.grad_norm([t.double()])
    assert float(cg.grad_norm([t, t])) == pytest.approx(math.sqrt(128.0))      # reading twice is fine
