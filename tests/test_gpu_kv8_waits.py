"""The bounded waits of spec_kv8_attention: where a piece of the cache does not come, the call ends by itself and says so in its
workspace.  In the bounds-checked build a hook withholds the pieces; the first test runs the others in it, and the tests of the
8-bit cache again."""
import os
import subprocess
import sys

import pytest
import torch

import speculative_decoding_verify_spec_gb300 as sv
from speculative_decoding_verify_spec_gb300 import _build, serve

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TIMEOUT, UNSUPPORTED = 4, 2


def test_under_the_checked_build():
    if os.environ.get("SV_CHECKS_ASSERT"):
        pytest.skip("already under the bounds-checked build")
    assert serve.lose_unit(0) == UNSUPPORTED
    env = dict(os.environ, SV_LIBRARY=_build.build_library(checks=True), SV_CHECKS_ASSERT="1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", "-m", "gpu",
                        *[os.path.join("tests", f) for f in ("test_gpu_kv8_waits.py", "test_gpu_kv8.py", "test_gpu_kv8_attention.py")]],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=1200)
    assert r.returncode == 0, (r.stdout[-4000:] + "\n" + r.stderr[-2000:]).strip()
    assert int(r.stdout.strip().splitlines()[-1].split(" passed")[0].split()[-1]) >= 150


@pytest.mark.parametrize("lost", [0, 1, 4])
@pytest.mark.parametrize("D,T,G,rope", [(64, 1, 4, False), (128, 6, 4, True), (128, 9, 4, False), (256, 4, 4, False), (64, 40, 4, False),
                                        (128, 40, 4, True), (256, 40, 4, False)])
def test_a_wait_that_runs_out(D, T, G, rope, lost):
    if not os.environ.get("SV_CHECKS_ASSERT"):
        pytest.skip("needs the bounds-checked build")
    g = torch.Generator().manual_seed(D)
    B, H, page, L = 700, 2, 64, 300  # several units a block, of several segments
    width = (L + T) // page + 1
    cache = torch.zeros((width, H, sv.spec_kv8_page_bytes(page, D)), dtype=torch.uint8, device=DEV)
    table = torch.arange(width, dtype=torch.int32, device=DEV).expand(B, width)
    start = torch.full((B,), L, dtype=torch.int32, device=DEV)
    k = torch.randn((1, L + T, H, D), generator=g).half().to(DEV)
    sv.spec_kv8_append(k, k, cache, table[:1], torch.zeros(1, dtype=torch.int32, device=DEV))
    q = torch.randn((B, T, H * G, D), generator=g).half().to(DEV)
    cos, sin = (torch.ones((1, D // 2), device=DEV), torch.zeros((1, D // 2), device=DEV)) if rope else (None, None)
    ws = torch.full((sv.spec_kv8_attention_workspace_size(B, T, H * G, H, D),), 0xA5, dtype=torch.uint8, device=DEV)

    def call():
        out = sv.spec_kv8_attention(q, cache, table, start, cos=cos, sin=sin, workspace=ws)
        return out, int(ws[:4].view(torch.int32)[0])

    want, status = call()
    assert status == 0
    try:
        assert serve.lose_unit(lost) == 0
        assert call()[1] == TIMEOUT
    finally:
        assert serve.lose_unit(-1) == 0
    again, status = call()  # the context is as it was
    assert status == 0 and torch.equal(again, want)
