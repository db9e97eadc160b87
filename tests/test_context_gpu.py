"""A caller's own CUDA context stays the current one: entry points bind the
device's primary context only to a thread that has none."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# A call without rows ends behind the check of the device, before any launch.
PROGRAM = """
import ctypes
cu = ctypes.CDLL("libcuda.so.1")
def call(name, *args):
    r = getattr(cu, name)(*args)
    assert r == 0, (name, r)
def current():
    c = ctypes.c_void_p()
    call("cuCtxGetCurrent", ctypes.byref(c))
    return c.value
call("cuInit", 0)
mine, dev = ctypes.c_void_p(), ctypes.c_int()
call("cuDeviceGet", ctypes.byref(dev), 0)
from deterministic_invariant_gemm_fwd_gb300 import _binding as b
call("cuCtxCreate_v2", ctypes.byref(mine), 0, dev)
assert current() == mine.value
for _ in range(2):
    st = b.lib.carbon_linear_logp_fwd(None, None, None, None, None, None, None, None, 0, 8, 50, 0, 1.0, -100, None, 0, 1, None)
    assert st == 0, st
    assert current() == mine.value, "the caller's context is no longer current"
call("cuCtxPopCurrent_v2", ctypes.byref(ctypes.c_void_p()))
assert current() is None
st = b.lib.carbon_linear_logp_fwd(None, None, None, None, None, None, None, None, 0, 8, 50, 0, 1.0, -100, None, 0, 1, None)
assert st == 0 and current() not in (None, mine.value)
call("cuCtxDestroy_v2", mine)
print("ok")
"""


def test_the_callers_context_stays_current():
    env = dict(os.environ)
    env.pop("CARBON_FAULT", None)
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stderr[-2000:]
