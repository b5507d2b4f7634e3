"""spec_kv_append and spec_kv_attention against their formulas in 64 bits.

The append is exact: every byte of the cache is compared.  The attention's tolerance, from its
roundings: a rotated query to 11 bits moves a score by at most 2^-11 scale sum|q_d k_d| (an fp16 one is held
exactly, and a 16-bit query that is not rotated is exact), each weight to fp16 by 2^-11 of itself, the output by half a step of its type; fp32 sums
and exponentials stay below 2^-16 of the largest value."""
import numpy as np
import pytest
import torch

import speculative_decoding_verify_spec_gb300 as sv
from tests import serve_util as U

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def np64(t):
    return t.double().cpu().numpy()


def pool(B, width, H, page, D, g, extra=2):
    pages = B * width + extra
    cache = torch.randint(0, 256, (pages, H, page * (D + 8)), generator=g, dtype=torch.uint8)
    table = torch.randperm(pages, generator=g)[:B * width].reshape(B, width).to(torch.int32)
    return cache, table


def expected_append(cache, table, k, v, start, new, page):
    """The cache's bytes after appending rotated keys k and values v [B, T, H, D] float64."""
    want = cache.numpy().copy()
    pages, H, _ = want.shape
    B, T, _, D = k.shape
    held = []
    for i, x in enumerate((k, v)):
        code, s, z = U.quantise(x)
        live = np.arange(T)[None] < new[:, None]
        held.append(np.where(live[..., None, None], z.astype(np.float64) + s.astype(np.float64) * code, 0.0))
        for b in range(B):
            for t in range(int(new[b])):
                j = int(start[b]) + t
                if j >= table.shape[1] * page:
                    continue
                pg, slot = int(table[b, j // page]), j % page
                if not 0 <= pg < pages:
                    continue
                row = want[pg]
                at = np.array([U.place(page, D, bool(i), slot, d) for d in range(0, D, 2)]) // 2
                row[:, at] = code[b, t, :, 0::2] | (code[b, t, :, 1::2] << 4)
                o = page * D + i * 4 * page + slot * 4
                row[:, o:o + 2] = s[b, t].view(np.uint8).reshape(H, 2)
                row[:, o + 2:o + 4] = z[b, t].view(np.uint8).reshape(H, 2)
    return want, held


def check_append(k, v, cache, table, start, new, page, cos=None, sin=None, positions=None, interleaved=False):
    B, T, H, D = k.shape
    cap = table.shape[1] * page
    st = np.clip(start.numpy(), 0, cap)
    n = np.full(B, T) if new is None else np.clip(new.numpy(), 0, T)
    at = positions.numpy() if positions is not None else st[:, None] + np.arange(T)
    rot = U.rotate(np64(k), None if cos is None else cos.numpy(), None if sin is None else sin.numpy(), at, interleaved)
    want, held = expected_append(cache, table.numpy(), rot, np64(v), st, n, page)
    dev = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    got = dev(cache).clone()
    kv, vv = sv.spec_kv_append(k.to(DEV), v.to(DEV), got, dev(table), dev(start), new_lens=dev(new), cos=dev(cos), sin=dev(sin),
                               positions=dev(positions), interleaved=interleaved, return_values=True)
    a, b = got.cpu().numpy(), want
    # (NaN words may differ in their bits: compare those as numbers)
    diff = a != b
    assert not diff[:, :, :page * D].any()
    x, y = (z[:, :, page * D:].copy().view(np.float16) for z in (a, b))
    assert ((x.view(np.uint16) == y.view(np.uint16)) | (np.isnan(x) & np.isnan(y))).all()
    for t, h in ((kv, held[0]), (vv, held[1])):
        with np.errstate(all="ignore"):
            r = torch.from_numpy(h).float().to(t.dtype)  # z + s code in fp32 (one rounding), then to the type
        assert torch.equal(torch.nan_to_num(t.cpu(), nan=1.25), torch.nan_to_num(r, nan=1.25))
    again = dev(cache).clone()
    assert sv.spec_kv_append(k.to(DEV), v.to(DEV), again, dev(table), dev(start), new_lens=dev(new), cos=dev(cos), sin=dev(sin),
                             positions=dev(positions), interleaved=interleaved) is None
    assert torch.equal(again, got)
    return got


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("B,T,H,page,rotary,interleaved", [(1, 1, 1, 16, 0, False), (3, 5, 2, 16, 1.0, False), (2, 40, 3, 48, 1.0, True),
                                                          (4, 9, 8, 64, 0.5, False), (2, 17, 1, 1024, 0.25, True), (1, 33, 2, 32, 6 / 64, False)])
def test_append(dtype, D, B, T, H, page, rotary, interleaved):
    g = torch.Generator().manual_seed(D + T)
    width = (70 + T) // page + 1
    cache, table = pool(B, width, H, page, D, g)
    k = (torch.randn((B, T, H, D), generator=g) * torch.exp(torch.randn((1, 1, H, D), generator=g))).to(DT[dtype])
    v = torch.randn((B, T, H, D), generator=g).to(DT[dtype])
    start = torch.randint(0, 70, (B,), generator=g, dtype=torch.int32)
    new = torch.randint(0, T + 1, (B,), generator=g, dtype=torch.int32)
    pairs = int(rotary * D) // 2
    cos, sin = U.tables(70 + T, pairs) if pairs else (None, None)
    check_append(k, v, cache, table, start, new, page, cos, sin, None, interleaved)
    check_append(k, v, cache, table, start, None, page, cos, sin,
                 torch.randint(-5, 200, (B, T), generator=g, dtype=torch.int32) if pairs else None, interleaved)


def test_append_many_codes_are_exact():
    """A million codes, with ranges over many powers of two: what lies near a border is settled exactly."""
    g = torch.Generator().manual_seed(5)
    B, T, H, D, page = 4, 256, 8, 128, 64
    cache, table = pool(B, T // page + 1, H, page, D, g)
    k = (torch.randn((B, T, H, D), generator=g) * torch.exp(4 * torch.randn((B, T, H, 1), generator=g))).to(torch.bfloat16)
    v = (torch.randint(-40, 41, (B, T, H, D), generator=g) * torch.exp2(torch.randint(-12, 5, (B, T, H, 1), generator=g).float())).to(torch.bfloat16)
    cos, sin = U.tables(400, 64)
    check_append(k, v, cache, table, torch.tensor([0, 3, 17, 60], dtype=torch.int32), None, page, cos, sin)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_append_special_values(dtype):
    g = torch.Generator().manual_seed(6)
    B, T, H, D, page = 1, 12, 2, 64, 16
    cache, table = pool(B, 2, H, page, D, g)
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
        k[0, 6] *= 1e30  # beyond fp16: zero and scale saturate
    k = k.to(DT[dtype])
    cos, sin = U.tables(50, 32)
    check_append(k, k.flip(1), cache, table, torch.tensor([3], dtype=torch.int32), None, page)
    keep = k.clone()
    keep[0, 6] = 1.0  # (sums of saturating numbers are not this test's)
    check_append(keep, keep.flip(1), cache, table, torch.tensor([3], dtype=torch.int32), None, page, cos, sin)


def test_append_bad_pages_and_lengths_touch_nothing_else():
    g = torch.Generator().manual_seed(7)
    B, T, H, D, page = 6, 20, 2, 128, 16
    cache, table = pool(B, 3, H, page, D, g)
    k, v = (torch.randn((B, T, H, D), generator=g).to(torch.bfloat16) for _ in range(2))
    table[0, 1] = -1
    table[1, 0] = cache.shape[0]
    table[2, 2] = 2**31 - 1
    start = torch.tensor([10, 0, 40, -7, 1000, 47], dtype=torch.int32)  # clamped to [0, 48]; past the table: dropped
    check_append(k, v, cache, table, start, torch.tensor([20, -3, 99, 20, 20, 20], dtype=torch.int32), page)


def test_append_strides():
    g = torch.Generator().manual_seed(8)
    B, T, H, D, page = 2, 7, 4, 128, 32
    cache, table = pool(B, 2, H, page, D, g)
    start = torch.tensor([3, 30], dtype=torch.int32)
    cos, sin = U.tables(64, 64)
    qkv = torch.randn((B, T, 3 * H * D + 1), generator=g).to(torch.float16).to(DEV)
    args = (table.to(DEV), start.to(DEV))
    for off in (0, 1):  # a fused projection's slices: on the vector grid (rows of odd length: not), and off it
        k, v = (qkv[..., off + i * H * D:off + (i + 1) * H * D].unflatten(-1, (H, D)) for i in (1, 1 if off else 2))
        a, b = cache.to(DEV), cache.to(DEV)
        sv.spec_kv_append(k, v, a, *args, cos=cos.to(DEV), sin=sin.to(DEV))
        sv.spec_kv_append(k.contiguous(), v.contiguous(), b, *args, cos=cos.to(DEV), sin=sin.to(DEV))
        assert torch.equal(a, b)
    k = qkv[..., :H * D].unflatten(-1, (H, D)).transpose(1, 2).contiguous().transpose(1, 2)  # heads before tokens
    a, b = cache.to(DEV), cache.to(DEV)
    sv.spec_kv_append(k, k, a, *args)
    sv.spec_kv_append(k.contiguous(), k.contiguous(), b, *args)
    assert torch.equal(a, b)
    one = k[:, :1, :1].expand(B, T, H, D)  # broadcast
    sv.spec_kv_append(one, one, a, *args)
    sv.spec_kv_append(one.contiguous(), one.contiguous(), b, *args)
    assert torch.equal(a, b)


# ------------------------------------------------------------------------ attention


def filled(B, n, H, page, D, width, g):
    """A cache whose slots below n[b] hold quantised vectors, the rest of it bytes of all kinds (NaN scales too)."""
    cache, table = pool(B, width, H, page, D, g)
    cache[:, :, page * D:] = 255
    c = cache.numpy()
    for b in range(B):
        m = min(int(n[b]), width * page)
        k = (torch.randn((1, m, H, D), generator=g) + 3 * (torch.rand((1, 1, H, D), generator=g) < 0.05)).numpy().astype(np.float64)
        v = torch.randn((1, m, H, D), generator=g).numpy().astype(np.float64)
        c[:] = expected_append(cache, table[b:b + 1].numpy(), k, v, np.array([0]), np.array([m]), page)[0]
    return cache, table


def check_attention(q, cache, table, start, new, page, parent=None, cos=None, sin=None, positions=None, interleaved=False, scale=None, got=None):
    B, T, Hq, D = q.shape
    pages, H = cache.shape[:2]
    cap = table.shape[1] * page
    sc = U.sm_scale(D) if scale is None else float(np.float32(scale))
    dev = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    if got is None:
        ws = torch.full((max(16, sv.spec_kv_attention_workspace_size(B, T, Hq, H, D)),), 0xA5, dtype=torch.uint8, device=DEV)
        got = sv.spec_kv_attention(dev(q), dev(cache), dev(table), dev(start), new_lens=dev(new), parent=dev(parent), scale=scale,
                                   cos=dev(cos), sin=dev(sin), positions=dev(positions), interleaved=interleaved, workspace=ws)
        assert int(ws[:4].view(torch.int32)[0]) == 0
    st = np.clip(start.numpy(), 0, cap)
    nn = np.full(B, T) if new is None else np.clip(new.numpy(), 0, T)
    at = positions.numpy() if positions is not None else st[:, None] + np.arange(T)
    qr = U.rotate(np64(q), None if cos is None else cos.numpy(), None if sin is None else sin.numpy(), at, interleaved)
    see_new = U.lines(None if parent is None else parent.numpy(), T)
    for b in range(B):
        n = min(int(st[b] + nn[b]), cap)
        k, v, held = U.read_cache(cache.numpy(), table.numpy(), page, D, b, n, pages)
        see = np.zeros((T, n), bool)
        see[:, :st[b]] = True
        see[:, st[b]:] = see_new[:, :n - st[b]]
        see &= held[None]
        see[nn[b]:] = False
        with np.errstate(all="ignore"):
            want = U.attention(qr[b], k, v, see, sc)
        x = np64(got[b])
        fine = np.isfinite(want)
        assert (np.isnan(x) == np.isnan(want)).all() and fine[~np.isnan(want)].all()
        if n:
            ok = np.isfinite(k) & np.isfinite(v)
            vmax = np.abs(np.where(ok, v, 0)).max()
            kk = np.repeat(np.where(ok, np.abs(k), 0).max(0)[None], T, 0) if n else 0
            move = 0.0 if cos is None or q.dtype == torch.float16 else 2.0**-11 * abs(sc) * (np.abs(qr[b]) * np.repeat(kk, Hq // H, 1)).sum(-1).max()
            tol = vmax * (2.0**-11 + 2 * move + 2.0**-16) + np.abs(want) * U.half_step(q.dtype)
            assert (np.abs(x - want)[fine] <= tol[fine]).all(), float((np.abs(x - want) - tol)[fine].max())
        else:
            assert (x == 0).all()
    return got


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("B,T,H,G,page,L", [(1, 1, 1, 1, 16, 0), (1, 1, 2, 8, 16, 63), (2, 1, 1, 4, 16, 64), (3, 5, 2, 4, 48, 200),
                                            (2, 9, 1, 7, 32, 129), (2, 17, 2, 8, 64, 300), (1, 70, 1, 1, 128, 5)])
def test_attention_chain(dtype, D, B, T, H, G, page, L):
    g = torch.Generator().manual_seed(D * 7 + T + L)
    width = (L + T) // page + 2
    start = torch.randint(0, L + 1, (B,), generator=g, dtype=torch.int32)
    start[0] = L
    new = torch.randint(0, T + 1, (B,), generator=g, dtype=torch.int32)
    new[0] = T
    cache, table = filled(B, start + T, H, page, D, width, g)
    q = (2 * torch.randn((B, T, H * G, D), generator=g)).to(DT[dtype])
    check_attention(q, cache, table, start, None, page)
    cos, sin = U.tables(L + T, D // 4)
    check_attention(q, cache, table, start, new, page, None, cos, sin, None, T % 2 == 0)


@pytest.mark.parametrize("D,H,G,T,page", [(64, 2, 4, 16, 16), (128, 1, 8, 40, 64), (128, 2, 1, 9, 16), (256, 1, 2, 70, 32), (64, 1, 16, 64, 64)])
def test_attention_tree(D, H, G, T, page):
    g = torch.Generator().manual_seed(T)
    B, L = 3, 150
    width = (L + T) // page + 1
    start = torch.tensor([L, 0, 61], dtype=torch.int32)
    parent = torch.tensor([-1] + [int(torch.randint(max(0, i - 5), i, (1,), generator=g)) for i in range(1, T)], dtype=torch.int32)
    cache, table = filled(B, start + T, H, page, D, width, g)
    q = torch.randn((B, T, H * G, D), generator=g).to(torch.float16)
    check_attention(q, cache, table, start, None, page, parent)
    depth = torch.tensor([len(U.path_of(parent, i)) for i in range(T)])
    cos, sin = U.tables(L + T, D // 2)
    new = torch.tensor([T, T // 2, 1], dtype=torch.int32)
    check_attention(q, cache, table, start, new, page, parent, cos, sin, (start[:, None] + depth).to(torch.int32))
    parent[T // 3], parent[T // 2] = T + 5, -9  # malformed: their paths end there
    check_attention(q, cache, table, start, None, page, parent)


@pytest.mark.parametrize("D,G,dtype,rope", [(256, 8, "fp16", True), (256, 8, "bf16", True), (128, 8, "bf16", True), (64, 1, "fp16", False)])
def test_attention_largest_tree(D, G, dtype, rope):
    """1024 nodes: the tree's own tables beside the largest rings in shared memory."""
    g = torch.Generator().manual_seed(D)
    T, page, L = 1024, 128, 5
    start = torch.tensor([L], dtype=torch.int32)
    parent = torch.tensor([-1] + [int(torch.randint(0, i, (1,), generator=g)) for i in range(1, T)], dtype=torch.int32)
    cache, table = filled(1, start + T, 1, page, D, 9, g)
    q = torch.randn((1, T, G, D), generator=g).to(DT[dtype])
    cos, sin = U.tables(T + L, D // 2) if rope else (None, None)
    check_attention(q, cache, table, start, None, page, parent, cos, sin)


def test_attention_tree_of_a_chain_is_the_chain():
    g = torch.Generator().manual_seed(3)
    B, T, H, G, D, page, L = 2, 12, 2, 4, 128, 16, 90
    start = torch.tensor([L, 7], dtype=torch.int32)
    cache, table = filled(B, start + T, H, page, D, 7, g)
    q = torch.randn((B, T, H * G, D), generator=g).to(torch.bfloat16).to(DEV)
    a = sv.spec_kv_attention(q, cache.to(DEV), table.to(DEV), start.to(DEV))
    b = sv.spec_kv_attention(q, cache.to(DEV), table.to(DEV), start.to(DEV), parent=torch.arange(-1, T - 1, dtype=torch.int32).to(DEV))
    assert torch.equal(a, b)


def test_attention_bad_pages_and_lengths():
    g = torch.Generator().manual_seed(4)
    B, T, H, G, D, page = 6, 3, 2, 2, 128, 16
    start = torch.tensor([60, 100, -5, 500, 0, 77], dtype=torch.int32)
    cache, table = filled(B, torch.tensor([112] * B), H, page, D, 7, g)
    table[0, 1], table[1, 0], table[1, 6], table[5] = -1, cache.shape[0], 2**31 - 1, -7  # sequence 5 sees nothing
    q = torch.randn((B, T, H * G, D), generator=g).to(torch.bfloat16)
    out = check_attention(q, cache, table, start, torch.tensor([3, 3, 2, 3, 0, 99], dtype=torch.int32), page)
    assert (out[4] == 0).all() and (out[5] == 0).all()


def test_attention_masked_nan_does_not_spread():
    """A NaN token is seen by its descendants alone; the others keep their results."""
    g = torch.Generator().manual_seed(9)
    B, T, H, G, D, page, L = 1, 8, 1, 4, 64, 16, 40
    start = torch.tensor([L], dtype=torch.int32)
    cache, table = filled(B, start + T, H, page, D, 3, g)
    j = L + 3
    c = cache.numpy()
    o = page * D + (j % page) * 4
    c[int(table[0, j // page]), 0, o:o + 4] = 0xFF
    c[int(table[0, j // page]), 0, o + 4 * page:o + 4 * page + 4] = 0xFF
    parent = torch.tensor([-1, 0, 0, 1, 2, 3, 4, 5], dtype=torch.int32)
    q = torch.randn((B, T, H * G, D), generator=g).to(torch.float16)
    out = check_attention(q, cache, table, start, None, page, parent)
    assert torch.isnan(out).any(-1).any(-1)[0].tolist() == [False, False, False, True, False, True, False, True]
    q[0, 1, 2, 5], q[0, 2, 0, 0] = float("nan"), float("inf")
    out = sv.spec_kv_attention(q.to(DEV), cache.to(DEV), table.to(DEV), start.to(DEV), parent=parent.to(DEV))
    bad = torch.isnan(out).any(-1)[0].cpu()
    assert bad[1].tolist() == [False, False, True, False] and bad[2].tolist() == [True, False, False, False]
    assert not bad[0].any() and not bad[4].any()


@pytest.mark.parametrize("D,rope", [(64, False), (64, True), (128, False), (128, True), (256, False)])
def test_attention_many_rows_masks_nan_and_growing_scores(D, rope):
    """The kernel for many rows: a NaN token stays with its descendants, NaN and infinite queries with their rows, scores that
    grow along the context move the maximum in the middle, and rows past the new tokens are 0."""
    g = torch.Generator().manual_seed(D)
    B, T, H, G, page, L = 2, 40, 1, 4, 16, 200
    start = torch.tensor([L, 70], dtype=torch.int32)
    width = (L + T) // page + 1
    cache, table = pool(B, width, H, page, D, g)
    c = cache.numpy()
    c[:, :, page * D:] = 255
    for b in range(B):
        m = int(start[b]) + T
        k = torch.randn((1, m, H, D), generator=g).numpy().astype(np.float64) * np.linspace(0.1, 12, m)[None, :, None, None]
        v = torch.randn((1, m, H, D), generator=g).numpy().astype(np.float64) * np.exp(np.linspace(-6, 6, m))[None, :, None, None]
        c[:] = expected_append(cache, table[b:b + 1].numpy(), k, v, np.array([0]), np.array([m]), page)[0]
    parent = torch.tensor([-1] + [int(torch.randint(max(0, i - 4), i, (1,), generator=g)) for i in range(1, T)], dtype=torch.int32)
    q = torch.randn((B, T, H * G, D), generator=g).to(torch.float16)
    cos, sin = U.tables(L + T, D // 2) if rope else (None, None)
    check_attention(q, cache, table, start, torch.tensor([T, 23], dtype=torch.int32), page, parent, cos, sin)
    check_attention(q, cache, table, start, None, page, None, cos, sin)
    j = L + 7
    for o in (page * D + (j % page) * 4, page * D + (page + j % page) * 4):
        c[int(table[0, j // page]), 0, o:o + 4] = 0xFF
    out = check_attention(q, cache, table, start, None, page, parent, cos, sin)
    sees = torch.from_numpy(U.lines(parent.numpy(), T)[:, 7])
    assert torch.equal(torch.isnan(out[0]).any(-1).any(-1).cpu(), sees) and not torch.isnan(out[1]).any()
    q[1, 3, 2, 5], q[1, 4, 0, 0] = float("nan"), float("inf")
    q[1, 5] = 60000.0
    out = sv.spec_kv_attention(q.to(DEV), cache.to(DEV), table.to(DEV), start.to(DEV), parent=parent.to(DEV))
    bad = torch.isnan(out[1]).any(-1).cpu()
    assert bad[3].tolist() == [False, False, True, False] and bad[4].tolist() == [True, False, False, False]
    assert not bad[0].any() and not bad[6:].any()


@pytest.mark.parametrize("scale", [0.0, -0.3, 5.0, 1e-20])
def test_attention_scales(scale):
    g = torch.Generator().manual_seed(10)
    B, T, H, G, D, page = 2, 4, 1, 4, 128, 16
    start = torch.tensor([130, 3], dtype=torch.int32)
    cache, table = filled(B, start + T, H, page, D, 9, g)
    q = torch.randn((B, T, H * G, D), generator=g).to(torch.float16)
    check_attention(q, cache, table, start, None, page, scale=scale)
    check_attention((q * 1e-6).to(torch.bfloat16), cache, table, start, None, page, scale=scale)


def test_attention_value_magnitudes():
    """Weights are held relative to the values' largest scale: tiny and huge values, together too, keep their precision."""
    g = torch.Generator().manual_seed(12)
    H, D, page, n = 1, 64, 16, 200
    for low, high in ((1e-5, 1e-5), (3e4, 3e4), (1e-3, 1e4), (1e4, 1e-3)):
        cache, table = pool(1, 13, H, page, D, g)
        size = np.linspace(np.log(low), np.log(high), n)
        k, v = (torch.randn((1, n, H, D), generator=g).numpy().astype(np.float64) for _ in range(2))
        v *= np.exp(size)[None, :, None, None]
        cache.numpy()[:] = expected_append(cache, table.numpy(), k, v, np.array([0]), np.array([n]), page)[0]
        q = torch.randn((1, 1, 4, D), generator=g).to(torch.bfloat16)
        check_attention(q, cache, table, torch.tensor([n - 1], dtype=torch.int32), None, page)


def test_attention_long_context_is_split_and_joined():
    """A context that every thread block takes a share of, against the plain sum on the GPU in 64 bits."""
    g = torch.Generator().manual_seed(13)
    H, G, D, page, L, T = 2, 4, 128, 64, 70001, 5
    width = (L + T) // page + 1
    cache, table = pool(1, width, H, page, D, g)
    scales = torch.rand((width + 2, H, 2, page, 2), generator=g) * 0.2 + 0.1
    scales[..., 1] = -7.5 * scales[..., 0]
    cache[:, :, page * D:] = scales.to(torch.float16).view(torch.uint8).reshape(width + 2, H, -1)
    q = torch.randn((1, T, H * G, D), generator=g).to(torch.float16)
    start = torch.tensor([L], dtype=torch.int32)
    got = np64(sv.spec_kv_attention(q.to(DEV), cache.to(DEV), table.to(DEV), start.to(DEV)))[0]
    n = L + T
    rows = cache[table[0].long()].numpy().reshape(width, H, -1)
    at = [np.array([[U.place(page, D, bool(i), s, d) for d in range(D)] for s in range(page)]) for i in (0, 1)]
    meta = rows[:, :, page * D:].copy().view(np.float16).astype(np.float64).reshape(width, H, 2, page, 2)
    kv = []
    for i in (0, 1):
        code = (rows[:, :, at[i] // 2] >> (4 * (at[i] % 2)).astype(np.uint8)) & 15
        kv.append((meta[:, :, i, :, 1:] + meta[:, :, i, :, :1] * code).transpose(0, 2, 1, 3).reshape(width * page, H, D)[:n])
    see = np.concatenate([np.ones((T, L), bool), U.lines(None, T)], 1)
    want = U.attention(np64(q)[0], kv[0], kv[1], see, U.sm_scale(D))
    vmax = np.abs(kv[1]).max()
    assert (np.abs(got - want) <= vmax * (2.0**-11 + 2.0**-16) + np.abs(want) * 2.0**-11).all()


def test_attention_many_sequences_share_blocks():
    g = torch.Generator().manual_seed(14)
    B, T, H, G, D, page = 300, 2, 2, 2, 64, 16
    start = torch.randint(0, 100, (B,), generator=g, dtype=torch.int32)
    start[::7] = 0
    new = torch.randint(0, T + 1, (B,), generator=g, dtype=torch.int32)
    cache, table = pool(B, 7, H, page, D, g)
    scales = torch.rand((B * 7 + 2, H, 2, page, 2), generator=g) * 0.2 + 0.1
    scales[..., 1] = -7.5 * scales[..., 0]
    cache[:, :, page * D:] = scales.to(torch.float16).view(torch.uint8).reshape(B * 7 + 2, H, -1)
    q = torch.randn((B, T, H * G, D), generator=g).to(torch.bfloat16)
    check_attention(q, cache, table, start, new, page)


def test_append_then_attend_graph_streams_and_strides():
    g = torch.Generator().manual_seed(15)
    B, T, H, G, D, page = 3, 6, 2, 4, 128, 16
    start = torch.tensor([50, 0, 33], dtype=torch.int32)
    cache, table = filled(B, start, H, page, D, 5, g)
    cos, sin = U.tables(80, 64)
    fused = torch.randn((B, T, (G + 2) * H * D), generator=g).to(torch.bfloat16).to(DEV)
    q, k, v = (x.unflatten(-1, (-1, D)) for x in fused.split([G * H * D, H * D, H * D], -1))
    c, tb, st, cs, sn = (x.to(DEV) for x in (cache, table, start, cos, sin))

    def step(pool_, out=None, ws=None):
        sv.spec_kv_append(k, v, pool_, tb, st, cos=cs, sin=sn)
        return sv.spec_kv_attention(q, pool_, tb, st, cos=cs, sin=sn, out=out, workspace=ws)

    pool_ = c.clone()
    want = step(pool_)
    check_attention(q.cpu(), pool_.cpu(), table, start, None, page, None, cos, sin, got=want)
    assert torch.equal(want, step(pool_))  # the same bits again
    side, out, ws = torch.cuda.Stream(), torch.empty_like(want), torch.empty(sv.spec_kv_attention_workspace_size(B, T, H * G, H, D), dtype=torch.uint8, device=DEV)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(c.clone(), out, ws)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    pool2 = c.clone()
    with torch.cuda.graph(graph):
        step(pool2, out, ws)
    for _ in range(2):
        out.zero_()
        pool2.copy_(c)
        graph.replay()
        assert torch.equal(out, want)


def test_bindings_refuse():
    q = torch.zeros((1, 2, 4, 64), dtype=torch.bfloat16, device=DEV)
    cache = torch.zeros((3, 2, 16 * 72), dtype=torch.uint8, device=DEV)
    table, start = torch.zeros((1, 2), dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    k = q[:, :, :2]
    assert sv.spec_kv_attention(q[:0], cache, table[:0], start[:0]).shape == (0, 2, 4, 64)
    assert sv.spec_kv_append(k[:, :0], k[:, :0], cache, table, start) is None
    for bad in (lambda: sv.spec_kv_attention(q[:, :, :3], cache, table, start), lambda: sv.spec_kv_attention(q, cache[..., :-1], table, start),
                lambda: sv.spec_kv_attention(q, cache, table.long(), start), lambda: sv.spec_kv_attention(q, cache, table, start[:0]),
                lambda: sv.spec_kv_attention(q, cache, table, start, cos=torch.zeros((4, 32), device=DEV)),
                lambda: sv.spec_kv_attention(q, cache, table, start, parent=start), lambda: sv.spec_kv_append(k, q, cache, table, start),
                lambda: sv.spec_kv_append(q, q, cache, table, start), lambda: sv.spec_kv_append(k, k, cache.int(), table, start),
                lambda: sv.spec_kv_append(k, k, cache, table, start, k_values=k)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        sv.spec_kv_attention(q.float(), cache, table, start)
    with pytest.raises(sv.SpecVerifyError, match="status 5"):
        sv.spec_kv_attention(q, cache, table, start, workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
    with pytest.raises(sv.SpecVerifyError, match="status 2"):
        sv.spec_kv_attention(torch.zeros((1, 1, 2, 96), dtype=torch.bfloat16, device=DEV),
                             torch.zeros((3, 2, 16 * 104), dtype=torch.uint8, device=DEV), table, start)
