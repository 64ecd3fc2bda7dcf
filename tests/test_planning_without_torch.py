"""Planning needs numpy and the library alone: torch is not imported for it, and
need not be there."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import sys
{hide}
import numpy as np
from context_document_masked_gb300 import fcp
p = fcp.Plan([300, 1, 83, 128], 2, "perdoc")
assert p.stats()["T"] == 512 and sum(p.shard(j)["tokens"] for j in range(2)) == 512
idx = np.concatenate([p.query_indices(j) for j in range(2)])
assert sorted(idx.tolist()) == list(range(512))
assert p.device_image().nbytes == p.device_bytes()
assert fcp.workspace_bytes(fcp.dims(512, 4, 2, 64), p) > 0
assert fcp.rel_buckets(32, 128)[0] == 0
assert fcp.strerror(fcp.ERR_UNSUPPORTED)
assert sys.modules.get("torch") is None
"""


@pytest.mark.parametrize("hide", ["", "sys.modules['torch'] = None  # its import raises"], ids=["not imported", "not there"])
def test_plan(lib, hide):
    r = subprocess.run([sys.executable, "-c", CODE.format(hide=hide)], cwd=ROOT, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr


def test_tensors_are_checked_at_the_first_call(lib):
    """The first call of a process that takes a tensor refuses a wrong one like any other."""
    code = ("from context_document_masked_gb300 import fcp\n"
            "for f in (lambda: fcp.device_status([0]), lambda: fcp.round_bf16(None, None), lambda: fcp.merge(1, 2, 3, 4)):\n"
            "    try:\n        f()\n    except ValueError as e:\n        assert 'expected a torch.Tensor' in str(e)\n"
            "    else:\n        raise SystemExit('accepted')\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr
