"""The example's decoding loop over the 8-bit cache: append, attention, logit adjustment and verification together."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_speculation_emits_what_plain_decoding_emits():
    """Greedy verification keeps the target's own choices, so drafts change the pace alone."""
    import verify_step as ex
    prompt = torch.arange(10, dtype=torch.int32, device="cuda").repeat(4, 2) + 11 * torch.arange(4, dtype=torch.int32, device="cuda")[:, None]
    plain, n = ex.decode(ex.Model(seed=3, bits=8), prompt, steps=30, gamma=0, repetition=1.0)
    assert (n == 50).all()
    spec, m = ex.decode(ex.Model(seed=3, bits=8), prompt, steps=20, gamma=4, repetition=1.0)
    for b in range(4):
        k = min(int(n[b]), int(m[b]))
        assert k >= 40 and torch.equal(plain[b, :k], spec[b, :k])


def test_only_allowed_tokens_are_emitted():
    import verify_step as ex
    prompt = torch.full((4, 8), 5, dtype=torch.int32, device="cuda")
    even = torch.full((256 // 32,), 0x55555555, dtype=torch.int32, device="cuda")
    h, n = ex.decode(ex.Model(seed=1, bits=8), prompt, steps=12, gamma=3, allowed_words=even)
    for b in range(4):
        assert (h[b, 8:int(n[b])] % 2 == 0).all()
