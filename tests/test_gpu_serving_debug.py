"""The page calls and the planned packed calls through the debug build, whose kernels check every
index that they compute: the same results, and nothing reported."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.mark.parametrize("name,pick", [
    ("test_gpu_pages.py", ""), ("test_gpu_page_status.py", ""), ("test_gpu_rope.py", ""), ("test_gpu_append_scales.py", ""),
    ("test_gpu_varlen_planned.py", "planned_lengths or (planned and 48-True-150) or fp32 or (test_planned and 700) or captured"),
])
def test_bounds_checking_build(name, pick):
    if os.environ.get("FA_LIBRARY"):
        pytest.skip("already on a chosen build")
    env = dict(os.environ, FA_LIBRARY=os.path.join(os.path.dirname(HERE), "exact_io_aware_81_b200", "libfa_debug.so"))
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-k", pick, os.path.join(HERE, name)],
                       env=env, cwd=os.path.dirname(HERE), capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and " passed" in r.stdout, r.stdout[-2000:] + r.stderr[-1000:]
