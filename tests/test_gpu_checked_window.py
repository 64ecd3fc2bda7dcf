"""The checked build on windowed attention and the residual norm: the suites run
through the library whose kernels check every index that they read from a plan's
tables. All inputs are valid: every case passes with no error bit set."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_checked_build_passes_the_window_suites(cuda):
    from context_document_masked_gb300 import build as b
    b.build(checked=True)
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider",
                        "tests/test_gpu_window.py", "tests/test_gpu_residual_norm.py"],
                       env=dict(os.environ, FCP_DEVICE_CHECKS="1"), cwd=ROOT, capture_output=True, text=True, timeout=1800)
    tail = r.stdout[-3000:] + r.stderr[-2000:]
    print(tail)
    assert r.returncode == 0, tail
