"""The rotary, cache and decode cases once more under libfa_checks.so: the same ABI compiled with
FA_CHECKS, whose kernels check their direct memory accesses against their tensors' sizes and record
FA_ERR_BOUNDS in the device status word, which every case asserts to be clean.  In a child process,
because the library is chosen when it is first loaded."""
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_serving_cases_pass_under_the_index_checking_build():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    path = os.path.join(ROOT, "exact_io_aware_80_b200", "libfa_checks.so")
    assert os.path.exists(path), "libfa_checks.so is not built (python -m exact_io_aware_80_b200.build --checks)"
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu and not slow", "tests/test_gpu_serving.py"],
                       env=dict(os.environ, FA_LIBRARY="libfa_checks.so"), cwd=ROOT, capture_output=True, text=True,
                       timeout=600)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
    assert " passed" in r.stdout
