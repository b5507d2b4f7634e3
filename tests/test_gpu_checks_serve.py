"""The tests of the operators around the verification step, run again against the bounds-checked build
of the library (see test_gpu_checks.py): every index into a buffer the library sizes itself is checked
against its extent."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.gpu
def test_serving_operators_under_the_checked_build():
    if os.environ.get("SV_CHECKS_ASSERT"):
        pytest.skip("already under the bounds-checked build")
    from speculative_decoding_verify_spec_gb300 import _build
    env = dict(os.environ, SV_LIBRARY=_build.build_library(checks=True), SV_CHECKS_ASSERT="1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", "-m", "gpu",
                        *[os.path.join("tests", f) for f in ("test_gpu_adjust.py", "test_gpu_kv.py")]],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=1200)
    assert r.returncode == 0, (r.stdout[-4000:] + "\n" + r.stderr[-2000:]).strip()
    assert int(r.stdout.strip().splitlines()[-1].split(" passed")[0].split()[-1]) >= 140
