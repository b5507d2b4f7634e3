"""spec_kv8_attention where one token's probability, or one block's scale, is far above those of the tokens that make the result:
kv8_bounds.py gives what each output may be off by, in shares of what goes into it."""
import math

import pytest
import torch

import speculative_decoding_verify_spec_gb300 as sv
from tests import kv8_bounds
from tests import kv8_reference as R
from tests import serve_util as U
from tests.test_gpu_kv8 import DEV, DT, dev
from tests.test_gpu_kv8_attention import filled

pytestmark = pytest.mark.gpu

FEW, MANY = [(1, 4), (9, 4)], [(40, 4)]  # (new tokens, query heads a kv head): the two kernels


def held(k, v, page):
    """A cache that holds k and v [B, n, H, D], and its table."""
    B, n, H, D = k.shape
    width = (n + page - 1) // page
    cache = torch.randint(0, 256, (B * width, H, sv.spec_kv8_page_bytes(page, D)), generator=torch.Generator().manual_seed(1), dtype=torch.uint8).to(DEV)
    table = torch.arange(B * width, dtype=torch.int32, device=DEV).flip(0).reshape(B, width)
    sv.spec_kv8_append(dev(k.bfloat16()), dev(v.bfloat16()), cache, table, torch.zeros(B, dtype=torch.int32, device=DEV))
    return cache, table


def check(q, cache, table, start, page, cap, new=None, parent=None, cos=None, sin=None):
    """The tolerance itself is at most `cap` of the sum of p |v|, and a step of the type's smallest numbers."""
    q, start, new, parent, cos, sin = (dev(t) for t in (q, start, new, parent, cos, sin))
    got = sv.spec_kv8_attention(q, cache, table, start, new_lens=new, parent=parent, cos=cos, sin=sin)
    want, tol, size = kv8_bounds.attention(q, cache, table, start, page, new, parent, cos, sin)
    assert (tol <= cap * size + 2 * torch.finfo(q.dtype).smallest_normal * torch.finfo(q.dtype).eps).all()
    R.check(got, want, tol)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T,G", FEW + MANY)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("L", [17, 100, 300])
def test_a_sink_of_small_values(L, D, T, G, dtype):
    """A first token with nearly all of the probability, whose value is 0 or small: the others are the result."""
    g = torch.Generator().manual_seed(L + D + T)
    H, page = 2, 32
    n = L + T
    u = torch.randint(0, 2, (H, D), generator=g) * 2.0 - 1
    q = (u.repeat_interleave(G, 0) + 0.05 * torch.randn((1, T, H * G, D), generator=g)).to(DT[dtype])
    start = torch.tensor([L], dtype=torch.int32)
    for rest in (7e-3, 1e-4, 1e-6, 1e-9):
        for value in (0.0, 2.0**-7):
            k, v = 0.3 * torch.randn((1, n, H, D), generator=g), torch.randn((1, n, H, D), generator=g)
            k[:, 0] = math.log((n - 1) / rest) / math.sqrt(D) * u  # its score is that logarithm, the others' are about 0
            v[:, 0] *= value
            check(q, *held(k, v, page), start, page, 2.0**-6)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("G", [2, 16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("L", [5, 120])
def test_quiet_tokens_in_a_loud_block(L, D, G, dtype):
    """Drafts that other rows do not see share a block of 16 with tokens that these do, and are louder by the factor."""
    g = torch.Generator().manual_seed(L + D + G)
    T, H, page = 8, 2, 16
    parent = torch.tensor([-1, 0, 0, 1, 2, 3, 4, 5], dtype=torch.int32)
    start = torch.tensor([L], dtype=torch.int32)
    q = torch.randn((1, T, H * G, D), generator=g).to(DT[dtype])
    for loud in (8, 12) if dtype == "fp16" else (8, 14, 20, 38):
        k, v = torch.randn((2, 1, L + T, H, D), generator=g)
        v[:, L + 5:] *= 2.0**loud
        check(q, *held(k, v, page), start, page, 2.0**-6, parent=parent)


@pytest.mark.parametrize("T,G", FEW + MANY)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_blocks_of_all_loudnesses(D, T, G):
    """Every block of 16 has another loudness, 2^-36 to 2^36, and a probability as much smaller: all take part in the result."""
    g = torch.Generator().manual_seed(D + T)
    H, page, n = 2, 64, 208
    u = torch.randint(0, 2, (H, D), generator=g) * 2.0 - 1
    q = (u.repeat_interleave(G, 0) + 0.02 * torch.randn((1, T, H * G, D), generator=g)).bfloat16()
    loud = torch.randint(-36, 37, (n // 16,), generator=g).double().repeat_interleave(16)[None, :, None, None]
    k = 0.3 * torch.randn((1, n, H, D), generator=g) - (loud * math.log(2) / math.sqrt(D)).float() * u
    v = torch.randn((1, n, H, D), generator=g) * torch.exp2(loud).float()
    check(q, *held(k, v, page), torch.tensor([n - T], dtype=torch.int32), page, 2.0**-5)


@pytest.mark.parametrize("T,G", FEW + MANY)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_dimensions_of_all_sizes(D, T, G):
    """Values whose dimensions differ by up to 2^16: codes down to the smallest, and those that are 0."""
    g = torch.Generator().manual_seed(D + T)
    H, page, n = 2, 64, 150 + T
    q = torch.randn((1, T, H * G, D), generator=g).bfloat16()
    k, v = torch.randn((2, 1, n, H, D), generator=g)
    check(q, *held(k, v * torch.exp2(-(torch.arange(D) % 17).float()), page), torch.tensor([150], dtype=torch.int32), page, 2.0**-6)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D,T,G,L", [(64, 300, 1, 77), (64, 150, 4, 0), (128, 300, 1, 0), (128, 131, 2, 300), (256, 290, 1, 100), (256, 130, 3, 1)])
def test_long_chains(D, T, G, L, dtype):
    """More new tokens than a tile holds, over contexts that are no multiple of one: prompts taken in pieces."""
    g = torch.Generator().manual_seed(D + T)
    B, H, page = 2, 2, 48
    start = torch.tensor([L, L // 2], dtype=torch.int32)
    cache, table = filled(B, start + T, H, page, D, (L + T) // page + 1, g, 0.0)
    q = 0.3 * torch.randn((B, T, H * G, D), generator=g)
    check(q.to(DT[dtype]), cache, table, start, page, 2.0**-5, new=torch.tensor([T, T - 7], dtype=torch.int32))
    cos, sin = U.tables(L + T, D // 2)
    check(q.to(DT[dtype]), cache, table, start, page, 2.0**-5, cos=cos, sin=sin)
