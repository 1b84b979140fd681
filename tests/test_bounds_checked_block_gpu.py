"""The block operators' GPU tests once more under the bounds-checked build
(-DDCN_CHECK_BOUNDS), in a child process (the binding loads one library per
process): every call ends with dcn_core_sync_status, which reports a skipped
access.  The cases of more than 2^31 values are left to the ordinary build."""
import os
import subprocess
import sys

import pytest

from deformable_convolution_core_b200 import build as dcn_build
from tests.conftest import ROOT

pytestmark = pytest.mark.gpu


def test_block_operators_under_the_bounds_checked_build():
    lib = dcn_build.build(checked=True)
    files = [os.path.join(ROOT, "tests", f"test_{n}_gpu.py") for n in ("quantize_fp8", "block_norm", "linear_fp8")]
    res = subprocess.run([sys.executable, "-m", "pytest", "-x", "-q", "-m", "gpu", "-p", "no:cacheprovider",
                          "-k", "not 2_31", *files], env=dict(os.environ, DCN_CORE_LIBRARY=lib), cwd=ROOT,
                         capture_output=True, text=True, timeout=900)
    assert res.returncode == 0, res.stdout[-4000:] + res.stderr[-2000:]
