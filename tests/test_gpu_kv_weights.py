"""spec_kv_attention: the bits that a row's weights keep do not depend on values that the row does not see or that weigh next to
nothing in it, nor on how small its weights are.  Tolerances: kv_reference.py, from what each row sees."""
import pytest
import torch

import speculative_decoding_verify_spec_gb300 as sv
from tests import kv_reference as R
from tests import serve_util as U

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
# query heads a kv head, new tokens: tiles of 8, 16, 40 rows, and the kernel for many rows
ROWS = [(64, 1, 4), (64, 4, 4), (64, 8, 20), (128, 8, 1), (128, 4, 9), (128, 4, 20), (256, 4, 4), (256, 2, 20), (256, 2, 40)]


def held(k, v, page, gen):
    """A cache that holds k, v [n, H, D] as its one sequence, its page table, and n."""
    n, H, D = k.shape
    width = (n + page - 1) // page
    cache = torch.zeros((width, H, page * (D + 8)), dtype=torch.uint8, device=DEV)
    table = torch.randperm(width, generator=gen).to(torch.int32)[None].to(DEV)
    start = torch.zeros(1, dtype=torch.int32, device=DEV)
    sv.spec_kv_append(k[None].to(DEV), v[None].to(DEV), cache, table, start)
    return cache, table


def compare(q, cache, table, start, page, **kw):
    """As many sequences over the same pages as give every thread block several units."""
    n, H = start + q.shape[1], cache.shape[1]
    B = 2000 // (H * -(-n // 128)) + 1  # at most 608 blocks, units of at most 128 tokens
    start = torch.tensor([start], dtype=torch.int32, device=DEV)
    want, tol = R.attention(q, cache, table, start, page, **kw)
    many = {k: v.expand(B, -1) if k == "positions" else v for k, v in kw.items()}
    got = sv.spec_kv_attention(q.expand(B, -1, -1, -1), cache, table.expand(B, -1), start.expand(B), **many).double()
    worst = ((got - want).abs() / tol).amax().item()
    assert worst <= 1, worst


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D,G,T", [r for r in ROWS if r[2] > 1])
@pytest.mark.parametrize("size", [500, 15000])
def test_a_hidden_tokens_values_take_no_bits_from_the_others(D, G, T, dtype, size):
    """A leaf of the tree whose values are thousands of times the others': only its own row sees it."""
    g = torch.Generator().manual_seed(D + T)
    L, H, page = 700, 2, 32
    k, v = (torch.randn((L + T, H, D), generator=g) for _ in range(2))
    v[L + T - 1] *= size
    cache, table = held(k.half(), v.half(), page, g)
    parent = torch.tensor([-1] + [max(0, i - 2) for i in range(1, T)], dtype=torch.int32, device=DEV)
    q = torch.randn((1, T, H * G, D), generator=g).to(DT[dtype]).to(DEV)
    compare(q, cache, table, L, page, parent=parent)
    cos, sin = U.tables(L + T, D // 2, DEV)
    if dtype == "fp16":
        compare(q, cache, table, L, page, parent=parent, cos=cos, sin=sin)


@pytest.mark.parametrize("D,G,T", ROWS)
@pytest.mark.parametrize("at", [3, 900])
def test_a_token_of_no_weight_takes_no_bits_from_the_others(D, G, T, at):
    """One seen token with huge values, whose key is far from every query."""
    g = torch.Generator().manual_seed(D + T + at)
    L, H, page = 1500, 1, 64
    k, v = (torch.randn((L + T, H, D), generator=g) for _ in range(2))
    way = torch.randn(D, generator=g)
    k[at] = -4 * way  # scores of about -4 sqrt(D) below the others'
    v[at] *= 1e4
    v *= 2.0**-6
    cache, table = held(k.half(), v.half(), page, g)
    q = (way + 0.1 * torch.randn((1, T, H * G, D), generator=g)).half().to(DEV)
    compare(q, cache, table, L, page)


@pytest.mark.parametrize("D,G,T", ROWS)
def test_small_weights_beside_a_large_one(D, G, T):
    """The first token takes nearly all the weight and has small values; thousands of others make up the output."""
    g = torch.Generator().manual_seed(D + T)
    L, H, page = 4000, 1, 64
    k, v = (torch.randn((L + T, H, D), generator=g) for _ in range(2))
    way = torch.randn(D, generator=g)
    way *= D**0.5 / way.norm()
    k[0] = way * 11 / D**0.5
    v[0] *= 0.01
    cache, table = held(k.half(), v.half(), page, g)
    q = (way + 0.02 * torch.randn((1, T, H * G, D), generator=g)).half().to(DEV)
    compare(q, cache, table, L, page)


@pytest.mark.parametrize("D,G,T", ROWS)
def test_values_without_a_range(D, G, T):
    """Constant value vectors have the smallest scale, 2^-24: alone, among others, and beside slots whose scale is 0."""
    g = torch.Generator().manual_seed(D + T)
    L, H, page = 300, 1, 16
    k, v = (torch.randn((L + T, H, D), generator=g) for _ in range(2))
    q = torch.randn((1, T, H * G, D), generator=g).half().to(DEV)
    flat = torch.randn((L + T, H, 1), generator=g).expand(L + T, H, D)
    some = torch.rand(L + T, generator=g) < 0.5
    for values in (flat, torch.where(some[:, None, None], flat, v)):
        cache, table = held(k.half(), values.half(), page, g)
        compare(q, cache, table, L, page)
    empty = table[0, 5].item()
    cache[empty] = 0  # 16 tokens of scale and zero 0
    compare(q, cache, table, L, page)
    assert not sv.spec_kv_attention(q, torch.zeros_like(cache), table, torch.tensor([L], dtype=torch.int32, device=DEV)).any()
