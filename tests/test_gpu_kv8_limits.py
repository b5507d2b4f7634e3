"""The 8-bit cache's operators at the ends of their ranges: pools past 32 bits, no pages, no table, queries that are no numbers."""
import pytest
import torch

import speculative_decoding_verify_spec_gb300 as sv
from tests import serve_util as U
from tests.test_gpu_kv8 import DEV, dev
from tests.test_gpu_kv8_attention import filled

pytestmark = pytest.mark.gpu


def int32(*x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("D,H,page,T,G", [(64, 8, 128, 6, 4), (128, 4, 64, 9, 4), (256, 2, 48, 40, 4)])
def test_pools_past_32_bits(D, H, page, T, G):
    """The pages at the far end of a pool of more than 2^32 bytes hold, give back and attend to what the same pages of a small pool do."""
    g = torch.Generator().manual_seed(D)
    B, L = 2, 200
    width = (L + T) // page + 1
    page_bytes = H * sv.spec_kv8_page_bytes(page, D)
    pages = (1 << 32) // page_bytes + B * width + 2
    big = torch.zeros((pages, H, page * (2 * D + 1)), dtype=torch.uint8, device=DEV)
    small = torch.zeros((B * width, H, page * (2 * D + 1)), dtype=torch.uint8, device=DEV)
    order = torch.randperm(B * width, generator=g).reshape(B, width).to(torch.int32)
    far = pages - B * width
    assert far * page_bytes >= 1 << 32
    k, v = (dev(torch.randn((B, L + T, H, D), generator=g).to(torch.bfloat16)) for _ in range(2))
    q = dev(torch.randn((B, T, H * G, D), generator=g).to(torch.bfloat16))
    cos, sin = U.tables(L + T, D // 2, DEV)
    results = []
    for cache, table in ((small, dev(order)), (big, dev(order) + far)):
        sv.spec_kv8_append(k, v, cache, table, int32(0, 0), cos=cos, sin=sin)
        out = sv.spec_kv8_attention(q, cache, table, int32(L, L - 30), cos=cos, sin=sin)
        results.append((out, *sv.spec_kv8_read(cache, table, int32(0, 0), L + T)))
    assert torch.equal(big[far:], small) and results[0][1].any()
    for a, b in zip(*results):
        assert torch.equal(a, b)
    assert not big[:B * width].any()


@pytest.mark.parametrize("T", [1, 20])
def test_no_table_and_no_pages(T):
    """A table of no pages, or a pool of none: appends are dropped, rows read and attended to are 0."""
    B, H, G, D, page = 2, 2, 4, 128, 16
    g = torch.Generator().manual_seed(T)
    x = dev(torch.randn((B, T, H, D), generator=g).to(torch.float16))
    q = dev(torch.randn((B, T, H * G, D), generator=g).to(torch.float16))
    for pages, width in ((3, 0), (0, 2)):
        cache = torch.full((pages, H, page * (2 * D + 1)), 0x5A, dtype=torch.uint8, device=DEV)
        table = torch.zeros((B, width), dtype=torch.int32, device=DEV)
        held, _ = sv.spec_kv8_append(x, x, cache, table, int32(0, 5), return_values=True)
        assert held.shape == x.shape and torch.isfinite(held).all() and held.any()
        assert (cache == 0x5A).all()
        for t in sv.spec_kv8_read(cache, table, int32(0, 5), T, dtype=torch.float16):
            assert t.shape == x.shape and not t.any()
        assert not sv.spec_kv8_attention(q, cache, table, int32(0, 5)).any()


@pytest.mark.parametrize("T,G", [(3, 2), (9, 4), (40, 4)])
def test_a_query_that_is_no_number_is_its_own_row_only(T, G):
    g = torch.Generator().manual_seed(T)
    B, H, D, page = 2, 2, 128, 16
    start = torch.tensor([150, 33], dtype=torch.int32)
    cache, table = filled(B, start + T, H, page, D, 13, g)
    q = torch.randn((B, T, H * G, D), generator=g).to(torch.bfloat16)
    args = (cache, table, dev(start))
    want = sv.spec_kv8_attention(dev(q), *args)
    q[0, 1, 1, 5], q[1, 2, 3, 0] = float("nan"), float("inf")
    got = sv.spec_kv8_attention(dev(q), *args)
    for at in ((0, 1, 1), (1, 2, 3)):
        assert torch.isnan(got[at]).all()
        got[at] = want[at] = 0
    assert torch.equal(got, want)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("off", [8, 3])
def test_rows_off_the_32_byte_grid(interleaved, off):
    """Rows, angles and results on the 16-byte grid only (rows off that too) hold and give back what those on the 32-byte grid do."""
    g = torch.Generator().manual_seed(off)
    B, T, H, D, page = 2, 40, 2, 128, 16

    def shifted(x, n):
        room = torch.zeros(x.numel() + n, dtype=x.dtype, device=DEV)
        room[n:] = x.reshape(-1)
        return room[n:].view(x.shape)

    k, v = (dev(torch.randn((B, T, H, D), generator=g).to(torch.float16)) for _ in range(2))
    cos, sin = U.tables(T + 20, D // 2, DEV)
    table = torch.arange(B * 4, dtype=torch.int32, device=DEV).view(B, 4)
    results = []
    for move in (0, 1):
        cache = torch.zeros((B * 4, H, page * (2 * D + 1)), dtype=torch.uint8, device=DEV)
        x, y, c, s = (shifted(t, move * n) for t, n in ((k, off), (v, off), (cos, 4), (sin, 4)))
        hk, hv, rk, rv = (shifted(torch.zeros_like(k), move * 8) for _ in range(4))
        assert all((t.data_ptr() % 32 != 0) == bool(move) for t in (x, y, c, s, hk, hv, rk, rv))
        sv.spec_kv8_append(x, y, cache, table, int32(5, 20), cos=c, sin=s, interleaved=interleaved, return_values=True, k_values=hk, v_values=hv)
        sv.spec_kv8_read(cache, table, int32(5, 20), T, dtype=torch.float16, k=rk, v=rv)
        results.append((cache, hk, hv, rk, rv))
    assert results[0][1].any()
    for a, b in zip(*results):
        assert torch.equal(a, b)
