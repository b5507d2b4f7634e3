"""The operators around the verification step on the CPU: sizes, the cache's layout, and every
refusal, which comes before any work is enqueued (the pointers below are never followed)."""
import ctypes

import numpy as np
import pytest
import torch

import speculative_decoding_verify_spec_gb300 as sv
from speculative_decoding_verify_spec_gb300 import _build, serve
from tests import serve_util as U

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 5
A = 1 << 20  # an aligned, never followed address


@pytest.fixture(scope="module")
def lib():
    _build.build_library()
    return serve._library()


def test_page_bytes(lib):
    for D in (64, 128, 256):
        for page in (16, 48, 1024):
            assert sv.spec_kv_page_bytes(page, D) == page * (D + 8)  # two times D / 2 bytes of codes, 4 of scale and zero
    for page, D in ((0, 128), (8, 128), (20, 128), (1040, 128), (16, 96), (16, 512), (-16, 64)):
        assert sv.spec_kv_page_bytes(page, D) == 0


@pytest.mark.parametrize("page,D", [(16, 64), (48, 128), (32, 256)])
def test_layout_is_the_documented_one_and_a_bijection(lib, page, D):
    seen = set()
    for values in (0, 1):
        for t in range(page):
            for d in range(D):
                o = lib.spec_kv_code_offset(page, D, values, t, d)
                assert o == U.place(page, D, values, t, d)
                seen.add(o)
    assert seen == set(range(2 * page * D))
    for bad in ((page, D, 0, -1, 0), (page, D, 0, page, 0), (page, D, 1, 0, D), (page, D, 1, 0, -1), (page + 1, D, 0, 0, 0)):
        assert lib.spec_kv_code_offset(*bad) == -1


def test_attention_workspace_size(lib):
    size = sv.spec_kv_attention_workspace_size
    assert size(0, 1, 8, 8, 128) == size(1, 0, 8, 8, 128) == size(1, 1, 8, 3, 128) == size(1, 1, 8, 8, 96) == 0
    # two partial results per thread block: 8 rows of D floats, a maximum and a sum each
    assert size(1, 1, 8, 8, 128) >= 152 * 2 * 8 * (128 + 2) * 4
    assert size(1, 1, 8, 8, 128) == size(500, 1, 64, 8, 128)  # by the rows that share a head, not the batch
    assert size(1, 1, 8, 8, 128) < size(1, 2, 64, 8, 128) < size(1, 9, 32, 8, 128)
    assert size(4, 9, 32, 8, 128) % 256 == 0


def adjust(lib, **kw):
    a = dict(logits=A, bs=80, rs=16, out=A, obs=80, ors=16, dtype=0, B=2, rows=5, V=16, history=A, hs=10, lengths=A,
             prompt=A, drafts=A, parent=None, rep=A, freq=A, pres=A, bt=A, bv=A, nbias=3, allowed=A)
    a.update(kw)
    return lib.spec_logit_adjust(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), UNSUPPORTED), (dict(dtype=-1), UNSUPPORTED), (dict(B=-1), INVALID), (dict(rows=-1), INVALID),
    (dict(V=0), INVALID), (dict(V=(1 << 30) + 1), INVALID), (dict(nbias=-1), INVALID), (dict(nbias=4097), INVALID),
    (dict(rows=1026, bs=1 << 20, obs=1 << 20), INVALID), (dict(rows=1025, parent=A, bs=1 << 20, obs=1 << 20), INVALID),
    (dict(bs=-1), INVALID), (dict(rs=-16), INVALID), (dict(obs=-1), INVALID), (dict(hs=-1), INVALID),
    (dict(hs=(1 << 30) + 1), INVALID), (dict(logits=None), INVALID), (dict(out=None), INVALID), (dict(lengths=None), INVALID),
    (dict(parent=A, drafts=None), INVALID), (dict(bt=None), INVALID), (dict(bv=None), INVALID),
    (dict(out=2 * A, ors=15), INVALID), (dict(out=2 * A, obs=0), INVALID), (dict(rs=32), INVALID), (dict(bs=0), INVALID),
    (dict(logits=A + 2), INVALID), (dict(dtype=1, logits=A + 1, out=2 * A), INVALID),
    (dict(B=0, logits=None), OK), (dict(rows=0, out=None), OK)])
def test_adjust_refusals(lib, kw, status):
    assert adjust(lib, **kw) == status


def append(lib, **kw):
    a = dict(k=A, kb=1024, kt=512, kh=128, v=A, vb=1024, vt=512, vh=128, dtype=1, B=2, T=2, H=4, D=128, cache=A, pages=9, page=16,
             table=A, width=4, start=A, new=None, cos=A, sin=A, len=64, pairs=64, inter=0, pos=None, kv=None, vv=None)
    a.update(kw)
    return lib.spec_kv_append(*a.values(), None)


SHARED = [
    (dict(dtype=0), UNSUPPORTED), (dict(dtype=3), UNSUPPORTED), (dict(D=96), UNSUPPORTED), (dict(page=24), UNSUPPORTED),
    (dict(page=0), UNSUPPORTED), (dict(page=2048), UNSUPPORTED), (dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(H=0), INVALID),
    (dict(pages=-1), INVALID), (dict(width=-1), INVALID), (dict(width=1 << 27), INVALID), (dict(sin=None), INVALID),
    (dict(cos=None), INVALID), (dict(pairs=65), INVALID), (dict(pairs=0), INVALID), (dict(len=0), INVALID),
    (dict(cache=A + 8), INVALID), (dict(cache=None), INVALID), (dict(table=None), INVALID), (dict(start=None), INVALID),
    (dict(B=0, cache=None, start=None), OK), (dict(T=0), OK)]


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(k=A + 1), INVALID), (dict(kb=-1), INVALID), (dict(vh=-1), INVALID),
    (dict(kv=A + 2), INVALID), (dict(vv=A + 4), INVALID), (dict(T=1 << 30, H=4), INVALID)])
def test_append_refusals(lib, kw, status):
    assert append(lib, **kw) == status


def attend(lib, **kw):
    a = dict(q=A, qb=4096, qt=2048, qh=128, dtype=1, B=2, T=2, Hq=16, H=4, D=128, cache=A, pages=9, page=16, table=A, width=4,
             start=A, new=None, parent=None, scale=0.1, cos=A, sin=A, len=64, pairs=64, inter=0, pos=None, out=A, ws=A, n=1 << 40)
    a.update(kw)
    return lib.spec_kv_attention(*a.values(), None)


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(q=A + 1), INVALID), (dict(out=A + 8), INVALID), (dict(Hq=15), INVALID),
    (dict(Hq=0), INVALID), (dict(qt=-1), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(T=1025, parent=A), INVALID), (dict(T=1 << 28), INVALID), (dict(ws=None), WORKSPACE), (dict(ws=A + 8), WORKSPACE),
    (dict(n=1000), WORKSPACE)])
def test_attention_refusals(lib, kw, status):
    assert attend(lib, **kw) == status


def test_bindings_refuse_what_they_cannot_take(lib):
    x = torch.zeros((1, 2, 8))
    with pytest.raises(ValueError, match="CUDA"):
        sv.spec_logit_adjust(x)
    h = torch.zeros((1, 1, 2, 64), dtype=torch.bfloat16)
    cache = torch.zeros((1, 2, 16 * 72), dtype=torch.uint8)
    i = torch.zeros((1, 1), dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        sv.spec_kv_append(h, h, cache, i, i[0])
    with pytest.raises(ValueError, match="CUDA"):
        sv.spec_kv_attention(h, cache, i, i[0])


def test_reference_quantiser_error_is_half_a_step():
    """The 64-bit form that the GPU tests compare with: a value is at most half a scale (and the zero's
    and scale's own roundings) from what its code stands for."""
    g = np.random.default_rng(1)
    x = g.normal(size=(50, 128)) * np.exp(g.normal(size=(50, 1)) * 3)
    code, s, z = U.quantise(x)
    s, z = s.astype(np.float64), z.astype(np.float64)
    tol = s / 2 + np.abs(z) * 2.0**-11 + 15 * s * 2.0**-10 + 2.0**-20
    assert (np.abs(z + s * code - x) <= tol).all()
    assert ctypes.sizeof(ctypes.c_void_p) == 8


@pytest.mark.parametrize("D,Hq,T", [(64, 4, 1), (64, 16, 40), (128, 4, 2), (128, 16, 9), (256, 8, 1), (256, 16, 40)])
def test_attention_capacity_limit(lib, D, Hq, T):
    """Token counts are rounded up to units of at most 128 tokens in 31 bits, so a table may span 2^31 - 128 tokens.  (No
    workspace: what passes the size check is refused after it, whatever the machine.)"""
    most = (1 << 31) - 128
    for page in (16, 128):
        call = dict(D=D, Hq=Hq, T=T, pairs=D // 2, page=page, ws=None)
        assert attend(lib, width=most // page, **call) == WORKSPACE
        assert attend(lib, width=most // page + 1, **call) == INVALID
    assert attend(lib, D=D, Hq=Hq, T=T, pairs=D // 2, page=48, width=most // 48 + 1, ws=None) == INVALID
