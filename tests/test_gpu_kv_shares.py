"""spec_kv_attention where every thread block has several units and segments: each kernel's instantiations by rows and head size, against
the formula in 64 bits; running maxima that move in the middle of a share; contexts that all blocks share.  Tolerances:
kv_reference.py."""
import pytest
import torch

import speculative_decoding_verify_spec_gb300 as sv
from tests import kv_reference as R
from tests import serve_util as U

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
MOST_BLOCKS, UNIT = 608, 128  # four blocks on each of 152 SMs, tokens of the largest unit


def pool(lens, k, v, page, gen):
    """A cache that holds k, v [S, n, H, D] for the S sequences' first lens tokens, slots behind them full of NaN."""
    S, n, H, D = k.shape
    width = -(-n // page) + 1
    pages = S * width + 3
    cache = torch.full((pages, H, page * (D + 8)), 255, dtype=torch.uint8, device=DEV)
    table = torch.randperm(pages, generator=gen)[:S * width].reshape(S, width).to(torch.int32).to(DEV)
    sv.spec_kv_append(k.half().to(DEV), v.half().to(DEV), cache, table, torch.zeros(S, dtype=torch.int32, device=DEV),
                      new_lens=torch.tensor(lens, dtype=torch.int32, device=DEV))
    return cache, table


def compare(q, cache, table, start, page, new=None, positions=None, least=3, **kw):
    """The S sequences of q, repeated until the blocks have `least` units each or more; every repeat is compared."""
    S, T, H = q.shape[0], q.shape[1], cache.shape[1]
    units = int(((start + T + UNIT - 1) // UNIT).sum()) * H
    many = -(-least * MOST_BLOCKS // units)
    assert units * many >= least * MOST_BLOCKS
    want, tol = R.attention(q, cache, table, start, page, new=new, positions=positions, **kw)
    rep = lambda t: None if t is None else t.repeat(many, *[1] * (t.dim() - 1))  # noqa: E731
    got = sv.spec_kv_attention(rep(q), cache, rep(table), rep(start), new_lens=rep(new), positions=rep(positions), **kw)
    assert not torch.isnan(got).any()
    got = got.double().reshape(many, *q.shape)
    worst = ((got - want).abs() / tol).amax().item()
    assert worst <= 1, worst


# (head size, query heads a kv head, new tokens): one, two, .. 8-row columns a tile, several tiles, and the kernel for many rows
SHAPES = [(64, 8, 1), (64, 4, 4), (64, 8, 3), (64, 4, 8), (64, 4, 15), (64, 4, 40), (64, 1, 130), (128, 4, 1), (128, 4, 4), (128, 8, 3),
          (128, 4, 8), (128, 4, 9), (128, 5, 9), (128, 8, 7), (128, 4, 20), (128, 8, 33), (256, 4, 2), (256, 4, 4), (256, 6, 4), (256, 4, 8),
          (256, 4, 10), (256, 8, 8), (256, 4, 17), (256, 4, 40)]


@pytest.mark.parametrize("dtype,rope", [("bf16", False), ("bf16", True), ("fp16", False), ("fp16", True)])
@pytest.mark.parametrize("D,G,T", SHAPES)
def test_each_shape_over_several_units_a_block(D, G, T, dtype, rope):
    g = torch.Generator().manual_seed(D * 1000 + G * 50 + T)
    H, page = 2, 48 if T % 2 else 64
    start = torch.tensor([700, 0, 511, 130, 1025])
    S, n = len(start), int(start.max()) + T
    k = torch.randn((S, n, H, D), generator=g) + 3 * (torch.rand((1, 1, H, D), generator=g) < 0.04)
    v = torch.randn((S, n, H, D), generator=g)
    cache, table = pool((start + T).tolist(), k, v, page, g)
    q = torch.randn((S, T, H * G, D), generator=g).to(DT[dtype]).to(DEV)
    start = start.to(torch.int32).to(DEV)
    cos, sin = U.tables(n, D // 4 if T % 2 else D // 2, DEV) if rope else (None, None)
    new = torch.tensor([T, max(1, T // 2), T, 1, T - T // 3], dtype=torch.int32, device=DEV)
    compare(q, cache, table, start, page, new=new, cos=cos, sin=sin, interleaved=T % 3 == 0)
    if T > 1:
        parent = torch.tensor([-1] + [int(torch.randint(max(0, i - 6), i, (1,), generator=g)) for i in range(1, T)], dtype=torch.int32)
        depth = torch.tensor([len(U.path_of(parent, i)) for i in range(T)], dtype=torch.int32, device=DEV)
        compare(q, cache, table, start, page, parent=parent.to(DEV), cos=cos, sin=sin, positions=start[:, None] + depth)


@pytest.mark.parametrize("exact", [False, True])
@pytest.mark.parametrize("D,G,T", [(64, 4, 1), (64, 4, 9), (64, 4, 40), (128, 8, 1), (128, 4, 9), (128, 4, 40), (256, 4, 6), (256, 4, 40)])
def test_maxima_that_move_within_a_share(D, G, T, exact):
    """One token outweighs each of those before it by more than 2^8, by its score or by its values, at a place of its own in each
    sequence: the sums and the weights under way move, and what came before it still makes up much of the output."""
    g = torch.Generator().manual_seed(D + T)
    H, page, n = 1, 64, 900
    places = (70, 129, 200, 333, 511, 640, 777, 895)
    S = 2 * len(places)
    way = torch.randn(D, generator=g)
    way *= D**0.5 / way.norm()  # way . way / sqrt(D) is sqrt(D)
    k = 0.3 * torch.randn((S, n + T, H, D), generator=g)
    v = torch.randn((S, n + T, H, D), generator=g)
    for i, at in enumerate(places):
        k[2 * i, at] = way * 6.3 / D**0.5  # a weight of 2^9
        k[2 * i + 1, at], v[2 * i + 1, at] = 0, v[2 * i + 1, at] * 700
    cache, table = pool([n + T] * S, k, v, page, g)
    q = (way + 0.02 * torch.randn((S, T, H * G, D), generator=g)).half().to(DEV)
    start = torch.full((S,), n, dtype=torch.int32, device=DEV)
    cos, sin = None, None
    if exact:  # angles of no turn: fp16 queries of two parts
        cos, sin = torch.ones((1, D // 2), device=DEV), torch.zeros((1, D // 2), device=DEV)
    compare(q, cache, table, start, page, cos=cos, sin=sin)


@pytest.mark.parametrize("D,G,T", [(64, 4, 9), (64, 4, 40), (128, 8, 1), (128, 4, 40), (256, 4, 6), (256, 4, 40)])
def test_scores_and_values_that_grow_along_the_context(D, G, T):
    """The maximum moves again and again; values grow too, by e^12."""
    g = torch.Generator().manual_seed(D + T)
    H, page, n = 1, 32, 1100
    way = torch.randn(D, generator=g)
    way *= D**0.5 / way.norm()
    rise = torch.linspace(0, 60 / D**0.5, n + T)[None, :, None, None]  # scores up to 60
    k = way * rise + 0.3 * torch.randn((2, n + T, H, D), generator=g)
    v = torch.randn((2, n + T, H, D), generator=g) * torch.exp(torch.linspace(-8, 4, n + T))[None, :, None, None]
    k[1], v[1] = k[1].flip(0), v[1].flip(0)
    cache, table = pool([n + T] * 2, k, v, page, g)
    q = (way + 0.02 * torch.randn((2, T, H * G, D), generator=g)).half().to(DEV)
    compare(q, cache, table, torch.full((2,), n, dtype=torch.int32, device=DEV), page)


@pytest.mark.parametrize("D,H,G,T,L", [(64, 2, 4, 6, 70001), (128, 2, 4, 5, 70001), (128, 1, 8, 1, 90000), (256, 2, 4, 6, 40007), (64, 2, 4, 40, 30011),
                                       (128, 1, 4, 40, 30011), (256, 1, 4, 40, 20003)])
def test_no_part_of_a_long_context_is_lost(D, H, G, T, L):
    """All blocks share one context of evenly weighed tokens: the roundings of thousands of weights average out, far below what any
    one block's part makes up."""
    g = torch.Generator().manual_seed(L + T)
    page, n = 64, L + T
    width = -(-n // page)
    cache = torch.randint(0, 256, (width, H, page * (D + 8)), generator=g, dtype=torch.uint8)
    scales = torch.rand((width, H, 2, page, 2), generator=g) * 0.2 + 0.1
    scales[..., 1] = -7.5 * scales[..., 0]
    cache[:, :, page * D:] = scales.half().view(torch.uint8).reshape(width, H, -1)
    cache, table = cache.to(DEV), torch.randperm(width, generator=g).to(torch.int32)[None].to(DEV)
    q = (0.5 * torch.randn((1, T, H * G, D), generator=g)).half().to(DEV)
    start = torch.tensor([L], dtype=torch.int32, device=DEV)
    got = sv.spec_kv_attention(q, cache, table, start).double()
    units = -(-n * H * 4 // (64 * 152))  # a block's share at most: units of 64 tokens, two row tiles, one block an SM
    want, tol = R.attention(q, cache, table, start, page, units=units)
    assert ((got - want).abs() / tol).amax().item() <= 1
    # the part of one of 608 blocks, left out, moves the outputs by about this much
    assert tol.amax().item() < want.std().item() / 608**0.5
