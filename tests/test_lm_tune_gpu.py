"""The operators of fine-tuning and scoring together, as they would be used, and
under the bounds-checked library."""
import math
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import deterministic_invariant_gemm_fwd_gb300 as cg  # noqa: E402
from deterministic_invariant_gemm_fwd_gb300 import nn  # noqa: E402
from tests.test_lm_gpu import same_bits, status  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_no_access_out_of_bounds():
    lib = os.path.join(ROOT, "deterministic_invariant_gemm_fwd_gb300", "libcarbon_gemm_bounds.so")
    assert os.path.exists(lib), "the bounds-checked library is not built"
    r = subprocess.run([sys.executable, "-m", "tests.tune_bounds_driver"], cwd=ROOT, capture_output=True, text=True,
                       env=dict(os.environ, CARBON_GEMM_LIBRARY=lib), timeout=600)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]
    assert r.stdout.strip().endswith("ok")


def step(ids, tokens, tasks, advantage, table0, w0, a0, b0, gamma0, scales, dtype):
    """A policy's step over [sequences, length]: loss, gradients before and after
    clipping, their norm.  In float64 torch operations for dtype float64."""
    leaves = [t.to(dtype).clone().requires_grad_() for t in (table0, w0, a0, b0, gamma0)]
    table, w, a, b, gamma = leaves
    if dtype is torch.float64:
        h = table[ids]
        x = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + 1e-6) * gamma
        at = tasks.clamp(min=0)
        u = torch.einsum("slk,slkr->slr", x, a[at]) * torch.where(tasks >= 0, scales.double()[at], 0.0)[..., None]
        y = x @ w + torch.einsum("slr,slrn->sln", u, b[at])
        s = h + y
        s = s * torch.rsqrt((s * s).mean(-1, keepdim=True) + 1e-6) * gamma
        lp = torch.log_softmax(s @ table.t() / 0.9, -1)
        logp = lp.gather(-1, tokens.clamp(min=0)[..., None])[..., 0]
        entropy = -(lp.exp() * lp).sum(-1)
        keep = tokens >= 0
        logp, entropy = torch.where(keep, logp, 0.0), torch.where(keep, entropy, 0.0)
    else:
        h = nn.embedding(ids, table)
        x = nn.rms_norm(h, gamma)
        y = nn.lora_linear(x, w, a, b, tasks, scales)
        s, _ = nn.rms_norm(y, gamma, residual=h)
        logp, entropy = nn.linear_log_probs(s, table, tokens, temperature=0.9)
    loss = -((advantage * logp).sum() + 0.05 * entropy.sum()) / (tokens >= 0).sum()
    loss.backward()
    grads = [t.grad.clone() for t in leaves]
    if dtype is torch.float64:
        norm = math.sqrt(sum(float((g * g).sum()) for g in grads))
        return loss.detach(), grads, norm, [g * min(1.0, 0.5 / (norm + 1e-6)) for g in grads]
    norm = nn.clip_grad_norm_(leaves, 0.5)
    return loss.detach(), grads, norm, [t.grad for t in leaves]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "f16"])
def test_a_policy_step(dtype):
    g = torch.Generator(device="cuda").manual_seed(5)
    S, L, V, D, n, r = 9, 37, 701, 136, 3, 16

    def randn(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)
    ids = torch.randint(0, V, (S, L), generator=g, device="cuda")
    tokens = torch.randint(0, V, (S, L), generator=g, device="cuda")
    tokens[:, :7] = -100
    tasks = torch.randint(-1, n, (S, 1), generator=g, device="cuda").expand(S, L).contiguous()
    advantage = torch.randn(S, L, generator=g, device="cuda")
    args = (ids, tokens, tasks, advantage, randn(V, D, std=0.3), randn(D, D, std=1 / math.sqrt(D)),
            randn(n, D, r, std=1 / math.sqrt(D)), randn(n, r, D, std=0.5 / math.sqrt(r)), 1 + randn(D, std=0.1),
            torch.tensor([1.0, 0.5, 2.0], device="cuda"))
    one, two = step(*args, dtype), step(*args, dtype)
    assert status() == 0
    assert torch.equal(one[0], two[0]) and torch.equal(one[2], two[2])
    assert all(same_bits(p, q) for p, q in zip(one[1] + one[3], two[1] + two[3]))
    want = step(*args, torch.float64)
    # Eight roundings to `dtype` lie on a gradient's way (h, x, y, the stream, s, and
    # back through them), each of half a step relative to the row that it is in;
    # the products' sums of D and V terms add them up like independent errors, and
    # what is left of the entries' own signs at most doubles them.
    eps = torch.finfo(dtype).eps / 2
    assert abs(float(one[0] - want[0])) <= 16 * eps * (1.0 + abs(float(want[0])))
    for got, ref in ((one[1], want[1]), (one[3], want[3])):
        for p, q in zip(got, ref):
            assert float((p.double() - q).norm()) <= 16 * eps * float(q.norm()) + 1e-7 * math.sqrt(q.numel())
    assert abs(float(one[2]) - want[2]) <= 16 * eps * want[2]


def test_alternatives_are_the_tokens_log_probabilities():
    """Scoring the alternatives one by one gives their log probabilities again."""
    g = torch.Generator(device="cuda").manual_seed(6)
    for M in (40, 400):
        x, table = torch.randn(M, 72, generator=g, device="cuda").half(), torch.randn(900, 72, generator=g, device="cuda").half()
        t = torch.zeros(M, dtype=torch.long, device="cuda")
        r = cg.linear_log_probs_fwd(x, table, t, temperature=0.7, top=6)
        for k in range(6):
            each = cg.linear_log_probs_fwd(x, table, r.top_ids[:, k].contiguous(), temperature=0.7)
            assert torch.equal(each.log_probs, r.top_log_probs[:, k]) and torch.equal(each.entropy, r.entropy)


def test_adapters_in_a_decoding_step():
    """One token of each of many requests in one call: the bits of each request alone."""
    g = torch.Generator(device="cuda").manual_seed(7)
    n, K, N, r = 12, 264, 520, 16
    w, a, b = (torch.randn(*s, generator=g, device="cuda").bfloat16() * 0.05 for s in ((K, N), (n, K, r), (n, r, N)))
    x = torch.randn(50, K, generator=g, device="cuda").bfloat16()
    ids, scales = torch.randint(-1, n, (50,), generator=g, device="cuda"), torch.rand(n, generator=g, device="cuda")
    y = cg.lora_linear_fwd(x, w, a, b, ids, scales)
    for m in (0, 7, 23, 49):
        i = int(ids[m])
        one = cg.lora_linear_fwd(x[m:m + 1], w, a[max(i, 0):max(i, 0) + 1], b[max(i, 0):max(i, 0) + 1],
                                 torch.full((1,), min(i, 0), device="cuda"), scales[max(i, 0):max(i, 0) + 1].contiguous())
        assert same_bits(one, y[m:m + 1])


def test_examples():
    from examples import train_tied_lm, tune_adapters
    args = (601, 72, 3, 8, 6, 20, 3)
    one, two = tune_adapters.train(*args), tune_adapters.train(*args)
    assert one[:2] == two[:2] and all(math.isfinite(v) for pair in one[0] for v in pair)
    clipped = [train_tied_lm.train(301, 64, 1, 200, 3, clip=0.1) for _ in range(2)]
    assert clipped[0] == clipped[1] and clipped[0][1] != train_tied_lm.train(301, 64, 1, 200, 3)[1]


def test_example_gradients():
    """The example's adapters' gradients are those of the same policy in float64."""
    from examples import tune_adapters as ex
    torch.manual_seed(1)
    policy = ex.Policy(601, 72, 3, 8)
    with torch.no_grad():
        policy.layer.b.normal_(std=0.3)
    ids, tokens, task, advantage = ex.batch(601, 6, 20, 3, 0)
    logp, entropy = policy(ids, tokens, task)
    (-((advantage * logp).sum() + 0.01 * entropy.sum())).backward()
    table, w, bias = policy.embed.weight.double(), policy.layer.weight.double(), policy.layer.bias.double()
    a, b = (p.detach().double().requires_grad_() for p in (policy.layer.a, policy.layer.b))
    h = table[ids]
    x = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + 1e-6)
    at = task.clamp(min=0)
    u = torch.einsum("slk,slkr->slr", x, a[at]) * (task >= 0)[..., None]
    s = h + x @ w + bias + torch.einsum("slr,slrn->sln", u, b[at])
    s = s * torch.rsqrt((s * s).mean(-1, keepdim=True) + 1e-6)
    lp = torch.log_softmax(s @ table.t(), -1)
    keep = tokens >= 0
    got = torch.where(keep, lp.gather(-1, tokens.clamp(min=0)[..., None])[..., 0], 0.0)
    ent = torch.where(keep, -(lp.exp() * lp).sum(-1), 0.0)
    (-((advantage * got).sum() + 0.01 * ent.sum())).backward()
    eps = torch.finfo(torch.bfloat16).eps / 2
    for p, q in ((policy.layer.a.grad, a.grad), (policy.layer.b.grad, b.grad)):
        assert float((p.double() - q).norm()) <= 16 * eps * float(q.norm())
