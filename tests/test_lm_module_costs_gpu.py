"""The results of log probabilities are allocations of their own, and the
autograd form launches nothing beside the library's kernels but, for a gradient,
the copy of the entropy that its backward pass reads."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import deterministic_invariant_gemm_fwd_gb300 as cg  # noqa: E402
from deterministic_invariant_gemm_fwd_gb300 import nn  # noqa: E402
from tests.test_lm_gpu import gen, xent_case  # noqa: E402


def nodes(call):
    """The nodes of a graph of the call."""
    from ctypes import CDLL, byref, c_size_t, c_void_p
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        call()
    n = c_size_t()
    assert CDLL("libcuda.so.1").cuGraphGetNodes(c_void_p(graph.raw_cuda_graph()), None, byref(n)) == 0
    return n.value


def test_results_of_their_own():
    x, table, t = xent_case(33, 64, 300, "bf16", 1, kept=1.0)
    r = cg.linear_log_probs_fwd(x, table, t)
    assert len({v.untyped_storage().data_ptr() for v in r[:3]}) == 3
    X = x.clone().requires_grad_()
    lp, entropy = nn.linear_log_probs(X, table, t)
    assert torch.equal(lp, r.log_probs) and torch.equal(entropy, r.entropy)
    lp.mul_(2.0)                                             # a user may change them in place
    entropy.add_(1.0)
    assert torch.equal(nn.linear_log_probs(X, table, t)[1] + 1.0, entropy)
    lp.sum().backward()
    want = cg.linear_log_probs_bwd(torch.full((33,), 2.0, device="cuda"), None, x, table, t, r.lse)[0]
    assert torch.equal(X.grad, want)


def test_launches_beside_the_librarys():
    x, table, t = xent_case(32, 64, 300, "bf16", 2, kept=1.0)
    X = x.clone().requires_grad_()
    x3, X3, t3 = x.view(4, 8, 64), X.view(4, 8, 64), t.view(4, 8)
    nn.linear_log_probs(X, table, t)
    torch.cuda.synchronize()
    n = nodes(lambda: cg.linear_log_probs_fwd(x, table, t))
    assert nodes(lambda: nn.linear_log_probs(x, table, t)) == n == nodes(lambda: nn.linear_log_probs(x3, table, t3))
    assert nodes(lambda: nn.linear_log_probs(X, table, t)) == n + 1 == nodes(lambda: nn.linear_log_probs(X3, table, t3))


def test_results_of_any_shape():
    x, table, t = xent_case(24, 64, 300, "bf16", 3)
    r = cg.linear_log_probs_fwd(x, table, t, top=3)
    for shape in ((24,), (4, 6), (2, 3, 4), (24, 1)):
        X = x.view(*shape, 64).clone().requires_grad_()
        lp, entropy = nn.linear_log_probs(X, table, t.view(shape))
        with torch.no_grad():
            plain = nn.linear_log_probs(X, table, t.view(shape))
        assert lp.shape == entropy.shape == shape and not lp._is_view() and not entropy._is_view()
        assert torch.equal(lp, plain[0]) and torch.equal(entropy, plain[1]) and torch.equal(lp.flatten(), r.log_probs)
        entropy.zero_()                                      # what the backward pass reads is its own
        lp.sum().backward()
        best = nn.top_log_probs(X, table, t.view(shape), 3)
        assert best.top_ids.shape == (*shape, 3) and torch.equal(best.top_ids.view(24, 3), r.top_ids)
        assert best.lse.shape == shape and not best.log_probs.requires_grad
    one = nn.linear_log_probs(x[0], table, t.clamp(min=0)[0])      # a single position
    assert one[0].shape == () and float(one[0]) == float(cg.linear_log_probs_fwd(x[:1], table, t.clamp(min=0)[:1]).log_probs[0])
