"""spec_kv8_attention against its formula in 64 bits; kv8_reference.py derives the tolerances."""
import numpy as np
import pytest
import torch

import speculative_decoding_verify_spec_gb300 as sv
from tests import kv8_reference as R
from tests import serve_util as U
from tests.test_gpu_kv8 import DEV, DT, dev, pool

pytestmark = pytest.mark.gpu


def filled(B, n, H, page, D, width, g, strong=3.0):
    """A cache whose slots below n[b] hold vectors of several loudnesses, the rest of it bytes of all kinds (NaN codes and scales too)."""
    cache, table = pool(B, width, H, page, D, g)
    c = dev(cache)
    m = min(int(max(n)), width * page)
    loud = torch.exp2(torch.randint(-2, 3, (B, m // 16 + 1, 1, 1), generator=g).float()).repeat_interleave(16, 1)[:, :m]
    k = ((torch.randn((B, m, H, D), generator=g) + strong * (torch.rand((1, 1, H, D), generator=g) < 0.05)) * loud).to(torch.bfloat16)
    v = (torch.randn((B, m, H, D), generator=g) * loud.flip(1)).to(torch.bfloat16)
    lens = torch.as_tensor(n).clamp(0, m).to(torch.int32)
    sv.spec_kv8_append(dev(k), dev(v), c, dev(table), torch.zeros(B, dtype=torch.int32, device=DEV), new_lens=dev(lens))
    return c, dev(table)


def check(q, cache, table, start, new, page, parent=None, cos=None, sin=None, positions=None, interleaved=False, scale=None):
    B, T, Hq, D = q.shape
    q, start, new, parent, cos, sin, positions = (dev(t) for t in (q, start, new, parent, cos, sin, positions))
    ws = torch.full((max(16, sv.spec_kv8_attention_workspace_size(B, T, Hq, cache.shape[1], D)),), 0xA5, dtype=torch.uint8, device=DEV)
    got = sv.spec_kv8_attention(q, cache, table, start, new_lens=new, parent=parent, scale=scale, cos=cos, sin=sin, positions=positions,
                                interleaved=interleaved, workspace=ws)
    assert int(ws[:4].view(torch.int32)[0]) == 0
    want, tol = R.attention(q, cache, table, start, page, new, parent, cos, sin, positions, interleaved, scale)
    R.check(got, want, tol)
    return got


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("B,T,H,G,page,L", [(1, 1, 1, 1, 16, 0), (1, 1, 2, 8, 16, 127), (2, 1, 1, 4, 16, 128), (3, 5, 2, 4, 48, 300),
                                            (2, 9, 1, 7, 32, 129), (2, 17, 2, 8, 64, 300), (1, 70, 1, 1, 128, 5), (1, 2, 2, 6, 1024, 700)])
def test_chain(dtype, D, B, T, H, G, page, L):
    g = torch.Generator().manual_seed(D * 7 + T + L)
    width = (L + T) // page + 2
    start = torch.randint(0, L + 1, (B,), generator=g, dtype=torch.int32)
    start[0] = L
    new = torch.randint(0, T + 1, (B,), generator=g, dtype=torch.int32)
    new[0] = T
    cache, table = filled(B, start + T, H, page, D, width, g)
    q = (2 * torch.randn((B, T, H * G, D), generator=g)).to(DT[dtype])
    check(q, cache, table, start, None, page)
    cos, sin = U.tables(L + T, D // 4)
    check(q, cache, table, start, new, page, None, cos, sin, None, T % 2 == 0)


@pytest.mark.parametrize("D,H,G,T,page", [(64, 2, 4, 16, 16), (128, 1, 8, 40, 64), (128, 2, 1, 9, 16), (256, 1, 2, 70, 32), (64, 1, 16, 64, 64)])
def test_tree(D, H, G, T, page):
    g = torch.Generator().manual_seed(T)
    B, L = 3, 250
    width = (L + T) // page + 1
    start = torch.tensor([L, 0, 61], dtype=torch.int32)
    parent = torch.tensor([-1] + [int(torch.randint(max(0, i - 5), i, (1,), generator=g)) for i in range(1, T)], dtype=torch.int32)
    cache, table = filled(B, start + T, H, page, D, width, g)
    q = torch.randn((B, T, H * G, D), generator=g).to(torch.float16)
    check(q, cache, table, start, None, page, parent)
    depth = torch.tensor([len(U.path_of(parent, i)) for i in range(T)])
    cos, sin = U.tables(L + T, D // 2)
    new = torch.tensor([T, T // 2, 1], dtype=torch.int32)
    check(q, cache, table, start, new, page, parent, cos, sin, (start[:, None] + depth).to(torch.int32))
    parent[T // 3], parent[T // 2] = T + 5, -9  # malformed: their paths end there
    check(q, cache, table, start, None, page, parent)


@pytest.mark.parametrize("D,G,dtype,rope", [(256, 8, "fp16", True), (256, 8, "bf16", True), (128, 8, "bf16", True), (64, 1, "fp16", False)])
def test_largest_tree(D, G, dtype, rope):
    g = torch.Generator().manual_seed(D)
    T, page, L = 1024, 128, 5
    start = torch.tensor([L], dtype=torch.int32)
    parent = torch.tensor([-1] + [int(torch.randint(0, i, (1,), generator=g)) for i in range(1, T)], dtype=torch.int32)
    cache, table = filled(1, start + T, 1, page, D, 9, g)
    q = torch.randn((1, T, G, D), generator=g).to(DT[dtype])
    cos, sin = U.tables(T + L, D // 2) if rope else (None, None)
    check(q, cache, table, start, None, page, parent, cos, sin)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D,T,G", [(64, 1, 8), (64, 9, 4), (64, 16, 4), (64, 64, 4), (128, 1, 4), (128, 4, 5), (128, 9, 4), (128, 16, 4), (128, 40, 2), (256, 1, 8),
                                   (256, 6, 4), (256, 9, 4), (256, 20, 3), (256, 33, 4)])
def test_many_units_a_block(D, T, G, dtype):
    """Lengths of all kinds, so that a block's share holds several segments and the ends of others, and long ones that many share."""
    g = torch.Generator().manual_seed(D + T)
    B, H, page = 40, 3, 64
    L = 3000
    width = (L + T) // page + 1
    start = torch.cat([torch.randint(0, 400, (B - 4,), generator=g), torch.randint(L // 2, L + 1, (4,), generator=g)]).to(torch.int32)
    start[3], start[7] = 0, 128 - T
    new = torch.randint(0, T + 1, (B,), generator=g, dtype=torch.int32)
    new[-2:] = T
    cache, table = filled(B, start + T, H, page, D, width, g)
    q = torch.randn((B, T, H * G, D), generator=g).to(DT[dtype])
    cos, sin = U.tables(L + T, D // 2)
    check(q, cache, table, start, new, page, None, cos, sin)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D,T,G", [(64, 1, 4), (128, 9, 4), (256, 6, 4), (64, 17, 4), (128, 33, 2), (256, 70, 1)])
def test_one_long_context(D, T, G, dtype):
    """A sink at the start, whose weight is far above the others' together in a tile, and growing scores, so that maxima move."""
    g = torch.Generator().manual_seed(D)
    H, page, L = 2, 128, 40001
    width = (L + T) // page + 1
    cache, table = filled(1, [L + T], H, page, D, width, g, 0.0)
    q = torch.randn((1, T, H * G, D), generator=g)
    k = torch.randn((1, 1, H, D), generator=g)
    at = torch.zeros(1, dtype=torch.int32, device=DEV)
    sink = 3 * q[:, :1, ::G]  # scores of about 3 sqrt(D) from the first token's first head; keys after it are held as they were
    sv.spec_kv8_append(dev(sink.to(torch.bfloat16)), dev(k.to(torch.bfloat16)), cache, table, at)
    q = q.to(DT[dtype])
    st = torch.tensor([L], dtype=torch.int32)
    check(q, cache, table, st, None, page)
    check((0.25 * q.float()).to(DT[dtype]), cache, table, st, None, page)
    check(q, cache, table, st, None, page, scale=-0.5)
    check(q, cache, table, st, None, page, scale=0.0)


def test_a_tree_of_a_chain_is_the_chain():
    g = torch.Generator().manual_seed(3)
    B, T, H, G, D, page, L = 2, 12, 2, 4, 128, 16, 190
    start = torch.tensor([L, 7], dtype=torch.int32)
    cache, table = filled(B, start + T, H, page, D, 13, g)
    q = dev(torch.randn((B, T, H * G, D), generator=g).to(torch.bfloat16))
    a = sv.spec_kv8_attention(q, cache, table, dev(start))
    b = sv.spec_kv8_attention(q, cache, table, dev(start), parent=torch.arange(-1, T - 1, dtype=torch.int32).to(DEV))
    assert torch.equal(a, b)


def test_bad_pages_and_lengths():
    g = torch.Generator().manual_seed(4)
    B, T, H, G, D, page = 6, 3, 2, 2, 128, 16
    start = torch.tensor([160, 200, -5, 500, 0, 177], dtype=torch.int32)
    cache, table = filled(B, torch.tensor([208] * B), H, page, D, 13, g)
    cache[cache.shape[0] - 2:] = 255
    table[0, 1], table[0, 8], table[1, 0], table[1, 12], table[5] = -1, -1, cache.shape[0], 2**31 - 1, -7  # sequence 5 sees nothing
    q = torch.randn((B, T, H * G, D), generator=g).to(torch.bfloat16)
    out = check(q, cache, table, start, torch.tensor([3, 3, 2, 3, 0, 99], dtype=torch.int32), page)
    assert (out[4] == 0).all() and (out[5] == 0).all()


@pytest.mark.parametrize("T,G", [(8, 1), (8, 4), (8, 8), (8, 16)])
@pytest.mark.parametrize("what", ["key", "value"])
def test_masked_nan_does_not_spread(T, G, what):
    """A NaN token is seen by its descendants alone; the others keep their results."""
    g = torch.Generator().manual_seed(9)
    B, H, D, page, L = 1, 1, 64, 16, 140
    start = torch.tensor([L], dtype=torch.int32)
    cache, table = filled(B, start + T, H, page, D, 10, g)
    parent = torch.tensor([-1, 0, 0, 1, 2, 3, 4, 5], dtype=torch.int32)
    q = torch.randn((B, T, H * G, D), generator=g).to(torch.float16)
    k, v = (torch.randn((1, T, H, D), generator=g) for _ in range(2))
    (k if what == "key" else v)[0, 3, 0, 17] = float("nan")
    sv.spec_kv8_append(dev(k.half()), dev(v.half()), cache, table, dev(start))
    out = check(q, cache, table, start, None, page, parent)
    assert torch.isnan(out).all(-1).all(-1)[0].tolist() == [False, False, False, True, False, True, False, True]
    assert not torch.isnan(out[0, [0, 1, 2, 4, 6]]).any()
    q[0, 1, 0, 5], q[0, 2, 0, 0] = float("nan"), float("inf")
    out = sv.spec_kv8_attention(dev(q), cache, table, dev(start), parent=dev(parent))
    bad = torch.isnan(out).any(-1)[0].cpu()
    assert bad[1].tolist() == [True] + [False] * (G - 1) and bad[2].tolist() == [True] + [False] * (G - 1)
    assert not bad[0].any() and not bad[4].any()


def test_hidden_values_of_any_size_take_nothing():
    """Values that a row does not see, or that have no weight, however large, and keys whose scores overflow nothing."""
    g = torch.Generator().manual_seed(14)
    T, H, G, D, page, L = 8, 1, 2, 128, 16, 120
    start = torch.tensor([L], dtype=torch.int32)
    cache, table = filled(1, start + T, H, page, D, 9, g)
    k, v = torch.randn((2, 1, T, H, D), generator=g)
    v[0, 5:] *= 2.0**38  # (in the block of 16 that the earlier ones share)
    parent = torch.tensor([-1, 0, 0, 1, 2, 3, 4, 5], dtype=torch.int32)
    sv.spec_kv8_append(dev(k.bfloat16()), dev(v.bfloat16()), cache, table, dev(start))
    q = torch.randn((1, T, H * G, D), generator=g).to(torch.bfloat16)
    check(q, cache, table, start, None, page, parent)


@pytest.mark.parametrize("D,T,G", [(64, 3, 2), (128, 9, 4), (256, 2, 8)])
def test_strides_and_shared_workspace(D, T, G):
    g = torch.Generator().manual_seed(5)
    B, H, page = 3, 2, 32
    start = torch.tensor([250, 3, 100], dtype=torch.int32)
    cache, table = filled(B, start + T, H, page, D, 10, g)
    cos, sin = (dev(t) for t in U.tables(400, D // 2))
    x = torch.randn((B, T, 3 * H * G * D + 1), generator=g).to(torch.float16).to(DEV)
    ws = torch.empty(sv.spec_kv8_attention_workspace_size(B, T, H * G, H, D), dtype=torch.uint8, device=DEV)
    for off in (0, 1, D):
        q = x[..., off:off + H * G * D].unflatten(-1, (H * G, D))
        a = sv.spec_kv8_attention(q, cache, table, dev(start), cos=cos, sin=sin, workspace=ws)
        b = sv.spec_kv8_attention(q.contiguous(), cache, table, dev(start), cos=cos, sin=sin, workspace=ws)
        assert torch.equal(a, b)
    q = q.transpose(1, 2).contiguous().transpose(1, 2)
    out = torch.empty((B, T, H * G, D), dtype=torch.float16, device=DEV)
    assert torch.equal(sv.spec_kv8_attention(q, cache, table, dev(start), cos=cos, sin=sin, out=out), b) and torch.equal(out, b)
    with pytest.raises(sv.SpecVerifyError):
        sv.spec_kv8_attention(q, cache, table, dev(start), workspace=ws[:64])


def test_captured_with_an_append_on_a_side_stream():
    """A step in a graph, replayed with new inputs, and two graphs that share a workspace one after the other."""
    g = torch.Generator().manual_seed(6)
    B, T, H, G, D, page, L = 4, 5, 2, 4, 128, 16, 200
    cache, table = filled(B, [L] * B, H, page, D, 14, g)
    start = torch.tensor([150, 31, 0, 199], dtype=torch.int32, device=DEV)
    k, v = (dev(torch.randn((B, T, H, D), generator=g).bfloat16()) for _ in range(2))
    q = dev(torch.randn((B, T, H * G, D), generator=g).bfloat16())
    ws = torch.empty(sv.spec_kv8_attention_workspace_size(B, T, H * G, H, D), dtype=torch.uint8, device=DEV)
    out = torch.empty_like(q)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())

    def step():
        sv.spec_kv8_append(k, v, cache, table, start)
        sv.spec_kv8_attention(q, cache, table, start, workspace=ws, out=out)

    with torch.cuda.stream(stream):
        step()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step()
        graphs.append(graph)
    for i in range(4):
        k.copy_(torch.randn((B, T, H, D), generator=g).bfloat16())
        q.copy_(torch.randn((B, T, H * G, D), generator=g).bfloat16())
        torch.cuda.synchronize()
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        want, tol = R.attention(q, cache, table, start, page)
        R.check(out, want, tol)
    assert np.isfinite(out.float().cpu().numpy()).all()


def test_the_accepted_path_of_a_tree():
    """append (tree) - attention - read of the accepted path - append behind the context: as if the path alone had been appended."""
    g = torch.Generator().manual_seed(13)
    B, T, H, D, page, L = 2, 12, 2, 128, 16, 70
    cache, table = filled(B, [L] * B, H, page, D, 6, g)
    plain = cache.clone()
    start = torch.tensor([L - 6, 40], dtype=torch.int32, device=DEV)
    cos, sin = (dev(t) for t in U.tables(200, D // 2))
    parent = torch.tensor([-1, 0, 0, 1, 1, 2, 4, 4, 6, 0, 9, 8], dtype=torch.int32)
    path = torch.tensor([0, 1, 4, 6, 8])
    depth = torch.tensor([len(U.path_of(parent, i)) for i in range(T)])
    positions = (start[:, None] + dev(depth)).to(torch.int32)
    k, v = (dev(torch.randn((B, T, H, D), generator=g).clamp(-2, 2).bfloat16()) for _ in range(2))
    sv.spec_kv8_append(k, v, cache, table, start, cos=cos, sin=sin, positions=positions)
    q = dev(torch.randn((B, T, 2 * H, D), generator=g).bfloat16())
    tree = check(q, cache, table, start, None, page, parent, cos, sin, positions)
    tol = R.attention(q, cache, table, start, page, None, dev(parent), cos, sin, positions)[1][:, path]
    pk, pv = sv.spec_kv8_read(cache, table, start, len(path), slots=(start[:, None] + dev(path)).to(torch.int32))
    sv.spec_kv8_append(pk, pv, cache, table, start)
    sv.spec_kv8_append(k[:, path], v[:, path], plain, table, start, cos=cos, sin=sin)
    a, b = (sv.spec_kv8_read(c, table, torch.zeros_like(start), L, lens=start + len(path)) for c in (cache, plain))
    for x, y in zip(a, b):  # (the tree's block may have taken a larger scale: numbers below 2^-14 of it may differ)
        assert torch.allclose(x.float(), y.float(), rtol=0, atol=4 * 2.0**-9 * 2.0**-5)
    chain = check(q[:, path], cache, table, start, None, page, None, cos, sin)
    tol = tol + R.attention(q[:, path], cache, table, start, page, None, None, cos, sin)[1]
    assert ((tree[:, path].double() - chain.double()).abs() <= tol).all()
