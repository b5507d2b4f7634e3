"""spec_kv_append and spec_kv_attention at the ends of their ranges."""
import pytest
import torch

import speculative_decoding_verify_spec_gb300 as sv
from tests import serve_util as U

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("interleaved", [False, True])
def test_positions_past_31_bits_take_the_last_angles(interleaved):
    """A full table of 2^31 - 1024 tokens: the positions of the tokens behind it pass 2^31 on the way, and all lie past the
    angles' table.  (The tokens find no page; what they would be held as shows their rotation.)"""
    g = torch.Generator().manual_seed(21)
    T, D, page = 1500, 64, 1024
    width = (1 << 21) - 1
    cache = torch.zeros((1, 1, page * (D + 8)), dtype=torch.uint8, device=DEV)
    table = torch.full((1, width), -1, dtype=torch.int32, device=DEV)
    start = torch.tensor([width * page], dtype=torch.int32, device=DEV)
    cos, sin = U.tables(5, D // 2, DEV)
    k = torch.randn((1, 1, 1, D), generator=g).to(torch.bfloat16).to(DEV).expand(1, T, 1, D)
    got, _ = sv.spec_kv_append(k, k, cache, table, start, cos=cos, sin=sin, interleaved=interleaved, return_values=True)
    last = torch.full((1, T), 4, dtype=torch.int32, device=DEV)
    want, _ = sv.spec_kv_append(k, k, cache, table, start, cos=cos, sin=sin, interleaved=interleaved, positions=last, return_values=True)
    assert torch.equal(got, want)
    first, _ = sv.spec_kv_append(k, k, cache, table, start, cos=cos, sin=sin, interleaved=interleaved,
                                 positions=torch.zeros_like(last), return_values=True)
    assert not torch.equal(got, first) and not cache.any()
