"""Alternatives whose logits crowd the low entries, as frequent tokens do: where
lists are kept and a run over the first 2048 entries goes ahead (more than 256
positions, 16384 entries or more), against float64 and against calls of up to 256
positions, whose logits are stored."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import deterministic_invariant_gemm_fwd_gb300 as cg  # noqa: E402
from tests.test_lm_gpu import DT, gen, status  # noqa: E402
from tests.test_lm_logp_gpu import check_forward  # noqa: E402

# entries that lie in different blocks of 32 (of 16 classes) and of 128
SIX = [37, 261, 389, 645, 805, 933]
EIGHT = [32, 256, 384, 640, 800, 928, 1376, 1984]
KINDS, WIDTH = 16, 64


def crowded(M, V, dtype, seed):
    """x, table, tokens: position m is of kind m % 16, and the largest logits of a
    kind belong to entries planted for it.  The planted logits are 8 to 15.75 in
    steps of 1/4 and the sum of the other products, of size 1."""
    g = gen(seed)
    plain = WIDTH - KINDS
    x = torch.randn(M, WIDTH, generator=g, device="cuda")
    table = torch.randn(V, WIDTH, generator=g, device="cuda") * plain ** -0.5 / 4
    x[:, plain:], table[:, plain:] = 0.0, 0.0
    x[torch.arange(M, device="cuda"), plain + torch.arange(M, device="cuda") % KINDS] = 8.0
    for kind in range(KINDS):
        if kind < 2:
            at = torch.tensor((SIX, EIGHT)[kind], device="cuda")
        elif kind < 10:                                    # anywhere in the first 2048 entries
            at = torch.randperm(2048, generator=g, device="cuda")[:32]
        elif kind < 13:                                    # on both sides of the 2048th
            at = 1024 + torch.randperm(2048, generator=g, device="cuda")[:32]
        elif kind < 15:                                    # in runs, and the last ones
            at = torch.cat([2048 - 16 + torch.arange(24, device="cuda"), V - 8 + torch.arange(8, device="cuda")])
        else:
            at = torch.randperm(V, generator=g, device="cuda")[:32]
        order = torch.randperm(len(at), generator=g, device="cuda")
        table[at, plain + kind] = 1.0 + order.float() / 32
    tokens = (torch.rand(M, generator=g, device="cuda") ** 3 * V).long().clamp_(max=V - 1)
    tokens[torch.rand(M, generator=g, device="cuda") < 0.1] = -100
    return x.to(DT[dtype]), table.to(DT[dtype]), tokens


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,V", [(300, 16384), (300, 20001), (1100, 50257), (700, 2048 * 8 - 1)])
def test_low_entries_hold_the_largest_logits(M, V, dtype):
    x, table, t = crowded(M, V, dtype, M + V)
    for top in (1, 5, 6, 8, 9, 10, 14, 20, 28):
        check_forward(x, table, t, 1.0, top)


@pytest.mark.parametrize("top", [6, 8, 14, 20])
def test_the_number_of_positions_does_not_show(top):
    M, V = 600, 20000
    x, table, t = crowded(M, V, "bf16", 3)
    r = cg.linear_log_probs_fwd(x, table, t, top=top)
    for a, b in ((0, 1), (0, 256), (40, 140), (344, 600), (100, 400)):
        part = cg.linear_log_probs_fwd(x[a:b], table, t[a:b], top=top)
        assert all(torch.equal(p, q[a:b]) for p, q in zip(part, r))
    assert status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_equal_logits_with_a_run_ahead(dtype):
    M, V = 300, 20000
    g = gen(7)
    t = torch.zeros(M, dtype=torch.long, device="cuda")
    x = torch.randn(M, WIDTH, generator=g, device="cuda").to(DT[dtype])
    some = torch.randn(400, WIDTH, generator=g, device="cuda").to(DT[dtype])
    for top in (8, 28):
        check_forward(x, some.repeat(50, 1), t, 1.0, top)               # fifty of each, every 400 entries
        check_forward(x, some[:100].repeat_interleave(200, 0), t, 1.0, top)      # and side by side
        check_forward(torch.zeros_like(x), some.repeat(50, 1), t, 1.0, top)
