"""The operators around the linear layers under the bounds-checked library
(libcarbon_gemm_bounds.so): no kernel indexes outside its buffers
(tests/lm_bounds_driver.py, in a process of its own)."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_no_access_out_of_bounds():
    lib = os.path.join(ROOT, "deterministic_invariant_gemm_fwd_gb300", "libcarbon_gemm_bounds.so")
    assert os.path.exists(lib), "the bounds-checked library is not built"
    r = subprocess.run([sys.executable, "-m", "tests.lm_bounds_driver"], cwd=ROOT, capture_output=True, text=True,
                       env=dict(os.environ, CARBON_GEMM_LIBRARY=lib), timeout=600)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]
    assert r.stdout.strip().endswith("ok")
