"""A result of the cached attentions that a bounded wait gave up on: NaN throughout, also for a caller who gives no workspace and sees no status.
In the bounds-checked build a hook withholds pieces of the cache; the first test runs the others in it."""
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


def test_under_the_checked_build():
    if os.environ.get("SV_CHECKS_ASSERT"):
        pytest.skip("already under the bounds-checked build")
    env = dict(os.environ, SV_LIBRARY=_build.build_library(checks=True), SV_CHECKS_ASSERT="1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", "-m", "gpu", os.path.join("tests", "test_gpu_kv_given_up.py")],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, (r.stdout[-4000:] + "\n" + r.stderr[-2000:]).strip()
    assert int(r.stdout.strip().splitlines()[-1].split(" passed")[0].split()[-1]) >= 16


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D,B,T,G,H,L", [(64, 1, 1, 2, 1, 20), (128, 40, 9, 4, 2, 300), (128, 3, 40, 4, 2, 300), (256, 40, 1, 4, 2, 300)])
@pytest.mark.parametrize("bits", [4, 8])
def test_given_up(bits, D, B, T, G, H, L, dtype):
    if not os.environ.get("SV_CHECKS_ASSERT"):
        pytest.skip("needs the bounds-checked build")
    g = torch.Generator().manual_seed(D)
    page = 32
    width = (L + T + page - 1) // page
    size = sv.spec_kv_page_bytes(page, D) if bits == 4 else sv.spec_kv8_page_bytes(page, D)
    append, attention = (sv.spec_kv_append, sv.spec_kv_attention) if bits == 4 else (sv.spec_kv8_append, sv.spec_kv8_attention)
    cache = torch.zeros((width, H, size), dtype=torch.uint8, device=DEV)
    table = torch.arange(width, dtype=torch.int32, device=DEV).expand(B, width)
    start = torch.full((B,), L, dtype=torch.int32, device=DEV)
    k = torch.randn((1, L + T, H, D), generator=g).to(dtype).to(DEV)
    append(k, k, cache, table[:1], torch.zeros(1, dtype=torch.int32, device=DEV))
    q = torch.randn((B, T, H * G, D), generator=g).to(dtype).to(DEV)
    new = torch.full((B,), T, dtype=torch.int32, device=DEV)
    new[1:3] = 0  # (sequences without new tokens: zeros, but not then)
    want = attention(q, cache, table, start, new_lens=new)
    assert torch.isfinite(want).all() and want[0].any() and not want[1:3].any()
    try:
        assert serve.lose_unit(0) == 0
        assert torch.isnan(attention(q, cache, table, start, new_lens=new)).all()
    finally:
        assert serve.lose_unit(-1) == 0
    assert torch.equal(attention(q, cache, table, start, new_lens=new), want)
