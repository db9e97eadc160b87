"""Runs the operators around the linear layers on sizes that drive their index
arithmetic to the edges, and checks after every call that no kernel skipped an
access out of range.  Meant for the bounds-checked build: run it as
``CARBON_GEMM_LIBRARY=.../libcarbon_gemm_bounds.so python -m tests.lm_bounds_driver``
(tests/test_lm_bounds_gpu.py does).  Prints "ok" at the end."""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)


def main():
    import torch
    import deterministic_invariant_gemm_fwd_gb300 as cg
    from deterministic_invariant_gemm_fwd_gb300 import _binding

    lib = os.environ.get("CARBON_GEMM_LIBRARY", "")
    assert _binding.LIB_PATH == lib and lib, "CARBON_GEMM_LIBRARY must name the library under test"
    g = torch.Generator(device="cuda").manual_seed(1)

    def randn(*shape, dtype):
        return torch.randn(*shape, generator=g, device="cuda").to(dtype)

    def check(what):
        st = cg.carbon_get_device_status()
        assert st == 0, f"{what}: {cg.carbon_status_string(st)}"

    types = (torch.float32, torch.bfloat16, torch.float16)
    for M, V, D in ((1, 1, 1), (3, 2, 7), (17, 100, 24), (33, 31, 515), (8192, 300, 8), (8193, 50257, 40), (70001, 17, 3)):
        for dt in types:
            ids = (torch.rand(M, generator=g, device="cuda") ** 2 * V).long().clamp_(max=V - 1)
            cg.embedding_fwd(randn(V, D, dtype=dt), ids, 2.0)
            check(("embedding_fwd", M, V, D, dt))
            out = cg.embedding_bwd(randn(M, D, dtype=dt), ids, V, 2.0)
            cg.embedding_bwd(randn(M, D, dtype=dt), ids, V, padding_idx=V - 1, accumulate_to=out)
            check(("embedding_bwd", M, V, D, dt))
    for M, D in ((1, 1), (5, 3), (9, 257), (3000, 8), (700, 768), (33, 1027), (3, 4097), (7, 16384), (5, 16385)):
        for dt in types:
            x, gamma = randn(M, D, dtype=dt), randn(D, dtype=dt)
            for res in (None, randn(M, D, dtype=dt)):
                r = cg.rms_norm_fwd(x, gamma, res, quantize=True)
                cg.rms_norm_expand(r.codes, r.scales, gamma)
                cg.rms_norm_expand(r.codes, r.scales, dtype=dt)
                cg.rms_norm_bwd(x, gamma, r.rstd, h=r.h, dh=res)
                cg.rms_norm_bwd(x, gamma, r.rstd, codes=r.codes, scales=r.scales, dh=res, recompute=True)
                check(("rms_norm", M, D, dt))
    for M, D, V in ((1, 8, 1), (2, 64, 129), (130, 72, 257), (515, 264, 4097), (700, 768, 9001), (17000, 64, 300)):
        for dt in types[1:]:
            x, table = randn(M, D, dtype=dt), randn(V, D, dtype=dt) * 0.1
            t = torch.randint(0, V, (M,), generator=g, device="cuda")
            t[torch.rand(M, generator=g, device="cuda") < 0.3] = -100
            for red, grad in (("mean", torch.tensor(1.0, device="cuda")), ("none", torch.ones(M, device="cuda"))):
                _, lse = cg.linear_cross_entropy_fwd(x, table, t, reduction=red)
                check(("linear_cross_entropy_fwd", M, D, V, dt, red))
                cg.linear_cross_entropy_bwd(grad, x, table, t, lse, reduction=red)
                check(("linear_cross_entropy_bwd", M, D, V, dt, red))
    print("ok")


if __name__ == "__main__":
    main()
