"""spec_kv8_append and spec_kv8_read against their rule in 64 bits: every byte, every number."""
import numpy as np
import pytest
import torch

import speculative_decoding_verify_spec_gb300 as sv
from tests import kv8_reference as R
from tests import serve_util as U

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def np64(t):
    return t.double().cpu().numpy()


def dev(t):
    return None if t is None else t.to(DEV)


def pool(B, width, H, page, D, g, extra=2):
    """Pages of bytes of all kinds (scales of all kinds among them), and a page table."""
    pages = B * width + extra
    cache = torch.randint(0, 256, (pages, H, page * (2 * D + 1)), generator=g, dtype=torch.uint8)
    table = torch.randperm(pages, generator=g)[:B * width].reshape(B, width).to(torch.int32)
    return cache, table


def held_pool(B, width, H, page, D, g, loud=3):
    """The same with numbers for codes and scales of a few sizes, as appends leave them."""
    cache, table = pool(B, width, H, page, D, g)
    c = cache.numpy()
    codes = c[:, :, :2 * page * D]
    codes[(codes & 127) == 127] = 64
    codes[codes == 128] = 0
    n = c.shape[0] * H * page // 16
    e = torch.randint(-loud, loud + 1, (n, 2), generator=g).numpy() - 8
    words = np.zeros((n, 4), np.uint32)
    words[:, :2] = (e + 127) << 23
    words[::5, 0] |= 0x0011  # a few vectors held as NaN
    words[::7, 1] |= 0x8200
    c[:, :, 2 * page * D:] = words.view(np.uint8).reshape(c.shape[0], H, page)
    return cache, table


def check_append(k, v, cache, table, start, new, page, cos=None, sin=None, positions=None, interleaved=False):
    B, T, H, D = k.shape
    cap = table.shape[1] * page
    st = np.clip(start.numpy(), 0, cap)
    n = np.full(B, T) if new is None else np.clip(new.numpy(), 0, T)
    at = positions.numpy() if positions is not None else st[:, None] + np.arange(T)
    rot = U.rotate(np64(k), None if cos is None else cos.numpy(), None if sin is None else sin.numpy(), at, interleaved)
    want, held = R.append(cache.numpy(), table.numpy(), rot, np64(v), st, n, page)
    args = (dev(table), dev(start))
    kw = dict(new_lens=dev(new), cos=dev(cos), sin=dev(sin), positions=dev(positions), interleaved=interleaved)
    got = dev(cache).clone()
    kv, vv = sv.spec_kv8_append(dev(k), dev(v), got, *args, return_values=True, **kw)
    diff = np.argwhere(got.cpu().numpy() != want)
    assert not len(diff), [(tuple(i), int(got[tuple(i)]), int(want[tuple(i)]), int(cache[tuple(i)])) for i in diff[:5]]
    for t, h in ((kv, held[0]), (vv, held[1])):
        r = torch.from_numpy(h).to(t.dtype)  # (a code times a power of two: exact but for fp16's ends)
        assert torch.equal(torch.nan_to_num(t.cpu(), nan=1.25), torch.nan_to_num(r, nan=1.25))
    again = dev(cache).clone()
    assert sv.spec_kv8_append(dev(k), dev(v), again, *args, **kw) is None
    assert torch.equal(again, got)
    sv.spec_kv8_append(dev(k), dev(v), again, *args, **kw)  # the same once more changes nothing
    assert torch.equal(again, got)
    # what the cache holds for them, read back
    rk, rv = sv.spec_kv8_read(got, *args, T, lens=dev(new), dtype=k.dtype)
    there = np.zeros((B, T), bool)
    for b in range(B):
        for t in range(int(n[b])):
            j = int(st[b]) + t
            there[b, t] = j < cap and 0 <= int(table[b, j // page]) < cache.shape[0]
    there = torch.from_numpy(there).to(DEV)[..., None, None]
    for x, y in ((rk, kv), (rv, vv)):
        assert torch.equal(torch.nan_to_num(x, nan=1.25), torch.nan_to_num(torch.where(there, y, 0.0), nan=1.25))
    return got


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("B,T,H,page,rotary,interleaved", [(1, 1, 1, 16, 0, False), (3, 5, 2, 16, 1.0, False), (2, 40, 3, 48, 1.0, True),
                                                          (4, 9, 8, 64, 0.5, False), (2, 17, 1, 1024, 0.25, True), (1, 33, 2, 32, 6 / 64, False)])
def test_append(dtype, D, B, T, H, page, rotary, interleaved):
    g = torch.Generator().manual_seed(D + T)
    width = (70 + T) // page + 1
    k = (torch.randn((B, T, H, D), generator=g) * torch.exp(torch.randn((1, 1, H, D), generator=g))).to(DT[dtype])
    v = torch.randn((B, T, H, D), generator=g).to(DT[dtype])
    start = torch.randint(0, 70, (B,), generator=g, dtype=torch.int32)
    new = torch.randint(0, T + 1, (B,), generator=g, dtype=torch.int32)
    pairs = int(rotary * D) // 2
    cos, sin = U.tables(70 + T, pairs) if pairs else (None, None)
    cache, table = held_pool(B, width, H, page, D, g)
    check_append(k, v, cache, table, start, new, page, cos, sin, None, interleaved)
    cache, table = held_pool(B, width, H, page, D, g, loud=20)
    check_append(k, v, cache, table, start, None, page, cos, sin,
                 torch.randint(-5, 200, (B, T), generator=g, dtype=torch.int32) if pairs else None, interleaved)


def test_append_many_codes_are_exact():
    """A million codes over many powers of two, ties among them, and angles that cancel: what lies near a border is settled exactly."""
    g = torch.Generator().manual_seed(5)
    B, T, H, D, page = 4, 256, 8, 128, 64
    cache, table = held_pool(B, T // page + 1, H, page, D, g)
    k = (torch.randn((B, T, H, D), generator=g) * torch.exp(4 * torch.randn((B, T, H, 1), generator=g))).to(torch.bfloat16)
    v = (torch.randint(-40, 41, (B, T, H, D), generator=g) * torch.exp2(torch.randint(-12, 5, (B, T, H, 1), generator=g).float())).to(torch.bfloat16)
    cos, sin = U.tables(400, 64)
    start = torch.tensor([0, 3, 17, 60], dtype=torch.int32)
    check_append(k, v, cache, table, start, None, page, cos, sin)
    k[..., 64:] = k[..., :64]  # a cos - a sin: small beside its terms at 45 degrees
    cos[:], sin[:] = 0.5**0.5, 0.5**0.5 * (1 + torch.randn((400, 64), generator=g) * 2.0**-18)
    check_append(k, v, cache, table, start, None, page, cos, sin)
    cos[:], sin[:] = 1.0, 0.0  # not turned at all: ties
    check_append(v, k, cache, table, start, None, page, cos, sin)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_append_special_values(dtype):
    g = torch.Generator().manual_seed(6)
    B, T, H, D, page = 1, 24, 2, 64, 16
    cache, table = held_pool(B, 3, H, page, D, g)
    k = torch.randn((B, T, H, D), generator=g)
    k[0, 0] = 0
    k[0, 1] = 3.0
    k[0, 2, 0, 5] = float("nan")
    k[0, 3, 1, 60] = float("inf")
    k[0, 4, 0, 0] = float("-inf")
    k[0, 5] *= 1e-6
    k[0, 6] *= 1e4
    k[0, 7] = 60000.0
    k[0, 8, :, ::2] = -60000.0
    k[0, 9] = 1000 + 0.01 * k[0, 9]
    k[0, 10, :, 1:] = 0
    k[0, 11] = -0.0
    if dtype == "bf16":
        k[0, 12] *= 1e30  # beyond the scales: saturates
        k[0, 13] = 3e38
        k[0, 14] = 1e-38
    k[0, 15:] = 0  # a block of nothing
    k = k.to(DT[dtype])
    cos, sin = U.tables(50, 32)
    for start in (0, 3, 16):
        st = torch.tensor([start], dtype=torch.int32)
        check_append(k, k.flip(1), cache, table, st, None, page)
        check_append(k, k.flip(1), cache, table, st, None, page, cos, sin)
        check_append(k, k.flip(1), cache, table, st, None, page, 1.5 * cos, 1.5 * sin)  # (fp32 overflows for the largest)


def test_append_a_block_token_by_token():
    """Louder and louder tokens: each rounds its block's older ones to a larger scale; a quiet one leaves the scale; a new block starts anew."""
    g = torch.Generator().manual_seed(11)
    H, D, page, T = 2, 128, 32, 35
    cache, table = pool(1, 2, H, page, D, g)
    k = torch.randn((1, T, H, D), generator=g) * torch.exp2(torch.tensor([(5 * i) % 13 - 6.0 for i in range(T)]))[None, :, None, None]
    k = k.to(torch.bfloat16)
    got, want = cache.to(DEV), cache.numpy()
    for t in range(T):
        st = torch.tensor([t], dtype=torch.int32)
        sv.spec_kv8_append(k[:, t:t + 1].to(DEV), k[:, t:t + 1].to(DEV), got, table.to(DEV), st.to(DEV))
        want, _ = R.append(want, table.numpy(), np64(k[:, t:t + 1]), np64(k[:, t:t + 1]), [t], [1], page)
        assert (got.cpu().numpy() == want).all(), t
    a, _ = sv.spec_kv8_read(got, table.to(DEV), torch.zeros(1, dtype=torch.int32, device=DEV), T)
    # at most one rounding to 4 bits, and one at each of 13 doublings of the scale where a number is below 2^-14 of the block's largest
    x, y = np64(a), np64(k)
    largest = np.array([np.abs(y[0, i // 16 * 16:i // 16 * 16 + 16]).max() for i in range(T)])[:, None, None]
    assert (np.abs(x - y)[0] <= np.abs(y)[0] * 2.0**-4 + 14 * largest * 2.0**-17).all()


def test_append_over_dropped_drafts():
    """A step's tokens over those of an earlier step that were rejected: what is kept is kept."""
    g = torch.Generator().manual_seed(12)
    H, D, page = 2, 64, 16
    cache, table = held_pool(1, 3, H, page, D, g)
    k = torch.randn((1, 9, H, D), generator=g).to(torch.float16)
    st = torch.tensor([11], dtype=torch.int32)
    got = check_append(100 * k, k, cache, table, st, None, page).cpu()
    check_append(k, 50 * k, got, table, torch.tensor([13], dtype=torch.int32), None, page)
    check_append(k, k, got, table, torch.tensor([16], dtype=torch.int32), torch.tensor([0], dtype=torch.int32), page)


def test_append_bad_pages_and_lengths_touch_nothing_else():
    g = torch.Generator().manual_seed(7)
    B, T, H, D, page = 6, 20, 2, 128, 16
    cache, table = held_pool(B, 3, H, page, D, g)
    k, v = (torch.randn((B, T, H, D), generator=g).to(torch.bfloat16) for _ in range(2))
    table[0, 1] = -1
    table[1, 0] = cache.shape[0]
    table[2, 2] = 2**31 - 1
    start = torch.tensor([10, 0, 40, -7, 1000, 47], dtype=torch.int32)  # clamped to [0, 48]; past the table: dropped
    check_append(k, v, cache, table, start, torch.tensor([20, -3, 99, 20, 20, 20], dtype=torch.int32), page)


def test_append_strides():
    g = torch.Generator().manual_seed(8)
    B, T, H, D, page = 2, 7, 4, 128, 32
    cache, table = held_pool(B, 2, H, page, D, g)
    start = torch.tensor([3, 30], dtype=torch.int32)
    cos, sin = U.tables(64, 64)
    qkv = torch.randn((B, T, 3 * H * D + 1), generator=g).to(torch.float16).to(DEV)
    args = (table.to(DEV), start.to(DEV))
    for off in (0, 1):  # a fused projection's slices: on the vector grid (rows of odd length: not), and off it
        k, v = (qkv[..., off + i * H * D:off + (i + 1) * H * D].unflatten(-1, (H, D)) for i in (1, 1 if off else 2))
        a, b = cache.to(DEV), cache.to(DEV)
        sv.spec_kv8_append(k, v, a, *args, cos=cos.to(DEV), sin=sin.to(DEV))
        sv.spec_kv8_append(k.contiguous(), v.contiguous(), b, *args, cos=cos.to(DEV), sin=sin.to(DEV))
        assert torch.equal(a, b)
    k = qkv[..., :H * D].unflatten(-1, (H, D)).transpose(1, 2).contiguous().transpose(1, 2)  # heads before tokens
    a, b = cache.to(DEV), cache.to(DEV)
    sv.spec_kv8_append(k, k, a, *args)
    sv.spec_kv8_append(k.contiguous(), k.contiguous(), b, *args)
    assert torch.equal(a, b)
    one = k[:, :1, :1].expand(B, T, H, D)  # broadcast
    sv.spec_kv8_append(one, one, a, *args)
    sv.spec_kv8_append(one.contiguous(), one.contiguous(), b, *args)
    assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D,page,H", [(64, 48, 1), (128, 16, 3), (256, 64, 2)])
def test_read(dtype, D, page, H):
    g = torch.Generator().manual_seed(D)
    B, width = 5, 4
    cache, table = held_pool(B, width, H, page, D, g, loud=12)
    table[1, 2], table[2, 0] = -1, 10**6
    cap = width * page
    for T in (1, 7, 8, 33):
        start = torch.tensor([0, cap // 2 - 3, 5, -4, cap - 2], dtype=torch.int32)
        lens = torch.tensor([T, T + 3, T // 2, -1, T], dtype=torch.int32)
        slots = torch.randint(-3, cap + 3, (B, T), generator=g, dtype=torch.int32)
        for ln in (None, lens):
            for sl in (None, slots):
                k, v = sv.spec_kv8_read(dev(cache), dev(table), dev(start), T, lens=dev(ln), slots=dev(sl), dtype=DT[dtype])
                assert k.shape == v.shape == (B, T, H, D) and k.dtype == v.dtype == DT[dtype]
                for b in range(B):
                    n = T if ln is None else min(max(int(ln[b]), 0), T)
                    at = sl[b].tolist() if sl is not None else [min(max(int(start[b]), 0), cap) + t for t in range(T)]
                    (kc, ks), (vc, vs), there = R.read(cache, table, page, D, b, at)
                    there[n:] = False
                    for got, c, s in ((k, kc, ks), (v, vc, vs)):
                        want = torch.where(there[:, None, None], c * s, 0.0).to(DT[dtype])
                        assert torch.equal(torch.nan_to_num(got[b].cpu(), nan=1.25), torch.nan_to_num(want, nan=1.25))


def test_read_into_given_tensors_and_refusals():
    g = torch.Generator().manual_seed(3)
    cache, table = held_pool(2, 2, 2, 16, 64, g)
    c, t, st = cache.to(DEV), table.to(DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
    k, v = torch.empty((2, 2, 20, 2, 64), dtype=torch.float16, device=DEV)
    assert sv.spec_kv8_read(c, t, st, 20, k=k, v=v)[0] is k
    a, b = sv.spec_kv8_read(c, t, st, 20, dtype=torch.float16)
    assert torch.equal(a.nan_to_num(1.5), k.nan_to_num(1.5)) and torch.equal(b.nan_to_num(1.5), v.nan_to_num(1.5))
    assert sv.spec_kv8_read(c, t, st, 0)[0].shape == (2, 0, 2, 64)
    for bad in (dict(k=k[:, :19]), dict(k=k, v=v.bfloat16()), dict(lens=st[:1]), dict(slots=t)):
        with pytest.raises(ValueError):
            sv.spec_kv8_read(c, t, st, 20, **bad)
    with pytest.raises(TypeError):
        sv.spec_kv8_read(c, t, st, 20, dtype=torch.float32)
    with pytest.raises(ValueError, match="8-bit cache"):
        sv.spec_kv8_read(c[:, :, :-1].contiguous(), t, st, 20)
    with pytest.raises(ValueError, match="negative"):
        sv.spec_kv8_read(c, t, st, -1)


@pytest.mark.parametrize("interleaved", [False, True])
def test_positions_past_31_bits_take_the_last_angles(interleaved):
    """A full table of 2^31 - 1024 tokens: the positions of the tokens behind it pass 2^31 on the way, and all lie past the
    angles' table.  (The tokens find no page; what they would be held as shows their rotation.)"""
    g = torch.Generator().manual_seed(21)
    T, D, page = 1500, 64, 1024
    width = (1 << 21) - 1
    cache = torch.zeros((1, 1, page * (2 * D + 1)), dtype=torch.uint8, device=DEV)
    table = torch.full((1, width), -1, dtype=torch.int32, device=DEV)
    start = torch.tensor([width * page], dtype=torch.int32, device=DEV)
    cos, sin = U.tables(5, D // 2, DEV)
    k = torch.randn((1, 1, 1, D), generator=g).to(torch.bfloat16).to(DEV).expand(1, T, 1, D)
    kw = dict(cos=cos, sin=sin, interleaved=interleaved, return_values=True)
    got, _ = sv.spec_kv8_append(k, k, cache, table, start, **kw)
    last = torch.full((1, T), 4, dtype=torch.int32, device=DEV)
    want, _ = sv.spec_kv8_append(k, k, cache, table, start, positions=last, **kw)
    assert torch.equal(got, want)
    first, _ = sv.spec_kv8_append(k, k, cache, table, start, positions=torch.zeros_like(last), **kw)
    assert not torch.equal(got, first) and not cache.any()
    a, b = sv.spec_kv8_read(cache, table, start - 700, T)
    assert not a.any() and not b.any()
