"""Runs the operators of fine-tuning and scoring on sizes that drive their index
arithmetic to the edges, and checks after every call that no kernel skipped an
access out of range.  Meant for the bounds-checked build: run it as
``CARBON_GEMM_LIBRARY=.../libcarbon_gemm_bounds.so python -m tests.tune_bounds_driver``
(tests/test_lm_tune_gpu.py does).  Prints "ok" at the end."""
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

    def randn(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device="cuda").to(dtype)

    def check(what):
        st = cg.carbon_get_device_status()
        assert st == 0, f"{what}: {cg.carbon_status_string(st)}"

    halves = (torch.bfloat16, torch.float16)
    for M, D, V in ((1, 8, 1), (2, 64, 129), (130, 72, 257), (256, 64, 3001), (257, 64, 3001), (515, 264, 4097),
                    (3000, 64, 20000), (17000, 64, 300)):
        for dt in halves:
            x, table = randn(M, D, dtype=dt), randn(V, D, dtype=dt) * 0.1
            t = torch.randint(0, V, (M,), generator=g, device="cuda")
            t[torch.rand(M, generator=g, device="cuda") < 0.3] = -100
            for top in sorted({0, min(V, 8), min(V, 28)}):
                r = cg.linear_log_probs_fwd(x, table, t, top=top)
                check(("linear_log_probs_fwd", M, D, V, dt, top))
            grad = randn(M)
            cg.linear_log_probs_bwd(grad, grad, x, table, t, r.lse, r.entropy)
            check(("linear_log_probs_bwd", M, D, V, dt))
            cg.linear_log_probs_fwd(torch.zeros_like(x), table, t, top=min(V, 28))       # equal logits
            check(("linear_log_probs_fwd of zeros", M, D, V, dt))
    for M, K, N, n, r in ((1, 8, 8, 1, 8), (3, 64, 72, 2, 24), (64, 768, 264, 24, 16), (130, 136, 264, 5, 128),
                          (513, 72, 1032, 300, 8), (2100, 264, 328, 3, 72), (4100, 64, 72, 2, 16)):
        for dt in halves:
            x, w, dy = randn(M, K, dtype=dt), randn(K, N, dtype=dt), randn(M, N, dtype=dt)
            a, b, scales = randn(n, K, r, dtype=dt), randn(n, r, N, dtype=dt), torch.rand(n, generator=g, device="cuda")
            runs = torch.cumsum((torch.rand(M, generator=g, device="cuda") < 0.02).long(), 0) % (n + 1) - 1
            for ids in (torch.randint(-1, n, (M,), generator=g, device="cuda"), runs, torch.full_like(runs, -1)):
                _, u = cg.lora_linear_fwd(x, w, a, b, ids, scales, randn(N, dtype=dt), keep=True)
                check(("lora_linear_fwd", M, K, N, n, r, dt))
                cg.lora_linear_bwd(dy, x, w, a, b, ids, scales, u)
                check(("lora_linear_bwd", M, K, N, n, r, dt))
    for sizes in ([1], [7, 0, 9], [2047, 2049], [3] * 33, [257] * 300, [1000003, 5]):
        for shift in (0, 1, 3):
            grads = [randn(n + shift, dtype=(torch.float32, *halves)[i % 3])[shift:] for i, n in enumerate(sizes)]
            cg.clip_grads(grads, 0.5, out=[torch.empty_like(t) for t in grads])
            cg.clip_grads(grads, 0.5)
            check(("clip_grads", sizes[:3], shift))
    print("ok")


if __name__ == "__main__":
    main()
