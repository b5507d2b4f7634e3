"""The tests of the 8-bit cache's limits and of its attention's weights in the bounds-checked build, where an index outside its array is reported."""
import os
import subprocess
import sys

import pytest

from speculative_decoding_verify_spec_gb300 import _build

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("name,count", [("test_gpu_kv8_limits.py", 12), ("test_gpu_kv8_weights.py", 108)])
def test_under_the_checked_build(name, count):
    if os.environ.get("SV_CHECKS_ASSERT"):
        pytest.skip("already under the bounds-checked build")
    env = dict(os.environ, SV_LIBRARY=_build.build_library(checks=True), SV_CHECKS_ASSERT="1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", "-m", "gpu", os.path.join("tests", name)],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, (r.stdout[-4000:] + "\n" + r.stderr[-2000:]).strip()
    assert int(r.stdout.strip().splitlines()[-1].split(" passed")[0].split()[-1]) >= count
