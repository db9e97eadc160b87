"""Log probabilities of tokens that hold nearly all of the probability: never
above 0, entropies never below, and as near to float64 as the sums allow."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import deterministic_invariant_gemm_fwd_gb300 as cg  # noqa: E402
from tests.test_lm_gpu import DT, E, gen, status  # noqa: E402


def confident(M, V, size, lead, dtype, seed):
    """Logits that fp32 sums hold exactly (one product each, of 16-bit factors
    with few bits): multiples of 1/16 up to `size`, the token's `lead` above them."""
    g = gen(seed)
    x = torch.zeros(M, 8, device="cuda")
    x[:, 0] = torch.randint(1, 16, (M,), generator=g, device="cuda") / 16      # of the largest: size * 15 / 16
    table = torch.zeros(V, 8, device="cuda")
    table[:, 0] = torch.randint(0, 64, (V,), generator=g, device="cuda") * (size / 128)
    table[V // 2, 0] = size
    table[V // 2, 1], x[:, 1] = lead, 1.0
    t = torch.full((M,), V // 2, device="cuda")
    return x.to(DT[dtype]), table.to(DT[dtype]), t


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,V,size,lead,temperature", [
    (200, 1000, 64, 0, 1.0), (300, 3000, 64, 4, 0.7), (300, 129, 512, 0, 1.0), (500, 257, 512, 1, 0.1), (40, 20000, 64, 16, 1.3),
    (40, 1, 512, 0, 0.9), (400, 1, 64, 3, 1.0), (64, 2, 8, 0, 1e-3),
])
def test_sign_and_error(M, V, size, lead, temperature, dtype):
    x, table, t = confident(M, V, size, lead, dtype, M + V)
    top = min(5, V)
    r = cg.linear_log_probs_fwd(x, table, t, temperature=temperature, top=top)
    assert status() == 0
    assert bool((r.log_probs <= 0).all()) and bool((r.top_log_probs <= 0).all()) and bool((r.entropy >= 0).all())
    # the token is the first alternative, with the same bits
    assert torch.equal(r.top_ids[:, 0], t) and torch.equal(r.top_log_probs[:, 0], r.log_probs)
    z = x.double() @ table.double().t() / temperature
    lp = torch.log_softmax(z, 1)
    want = lp.gather(1, t[:, None])[:, 0]
    H = -(lp.exp() * lp).sum(1)
    # sums and exponentials; differences of logits are off by a few fp32 roundings and
    # by D 2^-30 of themselves, each weighed with its probability
    bound = (16 + math.log2(V)) * 2.0 ** -23 * (1 + want.abs() + H) + 8 * 2.0 ** -30 * (want.abs() + H) + 8 * E * H
    assert bool(((r.log_probs.double() - want).abs() <= bound).all()), float(((r.log_probs.double() - want).abs() / bound).max())


@pytest.mark.parametrize("M", [50, 700])
def test_not_a_number_stays(M):
    x, table, t = confident(M, 300, 64, 1, "bf16", 5)
    x[3, 4] = math.nan
    r = cg.linear_log_probs_fwd(x, table, t, top=3)
    rest = torch.arange(M, device="cuda") != 3
    assert bool(r.log_probs[3].isnan()) and bool(r.entropy[3].isnan()) and bool(r.lse[3].isnan())
    assert bool(r.log_probs[rest].isfinite().all())
    assert status() == 0
