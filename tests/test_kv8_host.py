"""The operators of the 8-bit paged cache on the CPU: sizes, the layout, the rule's own checks, and every refusal, which
comes before any work is enqueued (the pointers below are never followed)."""
import numpy as np
import pytest
import torch

import speculative_decoding_verify_spec_gb300 as sv
from speculative_decoding_verify_spec_gb300 import _build, serve
from tests import kv8_reference as R
from tests import test_serve_host as S

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 5
A = S.A


@pytest.fixture(scope="module")
def lib():
    _build.build_library()
    return serve._library()


def test_page_bytes(lib):
    seen = {}
    for D in (64, 128, 256):
        for page in range(16, 1025, 16):
            n = sv.spec_kv8_page_bytes(page, D)
            assert n == 2 * page * D + page  # two codes a dimension, 16 bytes a block of 16
            assert n % 16 == 0 and seen.setdefault(n, D) == D and serve._head_dim8(n) == D
    for page, D in ((0, 128), (8, 128), (20, 128), (1040, 128), (16, 96), (16, 512), (-16, 64)):
        assert sv.spec_kv8_page_bytes(page, D) == 0
    for n in (0, 16 * 129 + 1, 16 * (128 + 8), 2048 * 129):
        with pytest.raises(ValueError, match="8-bit cache"):
            serve._head_dim8(n)


@pytest.mark.parametrize("page,D", [(16, 64), (48, 128), (32, 256)])
def test_layout_is_the_documented_one_and_a_bijection(lib, page, D):
    seen = set()
    for values in (0, 1):
        for t in range(page):
            for d in range(D):
                o = lib.spec_kv8_code_offset(page, D, values, t, d)
                assert o == values * page * D + R.place(D, t, d)
                seen.add(o)
    assert seen == set(range(2 * page * D))
    for bad in ((page, D, 0, -1, 0), (page, D, 0, page, 0), (page, D, 1, 0, D), (page, D, 1, 0, -1), (page + 1, D, 0, 0, 0)):
        assert lib.spec_kv8_code_offset(*bad) == -1


def test_reference_codes():
    """The 64-bit form that the GPU tests compare with: every code is its own number's, and a number is held as the nearest code."""
    c = np.array([i for i in range(256) if i not in (127, 128, 255)])
    assert (R.code(R.NUMBERS[c]) == c).all()
    y = np.random.default_rng(1).normal(size=20000) * 2.0 ** np.random.default_rng(2).integers(-14, 9, 20000)
    near = np.abs(R.NUMBERS[c][None] - np.clip(y, -448, 448)[:, None]).min(1)
    assert (np.abs(R.NUMBERS[R.code(y)] - np.clip(y, -448, 448)) == near).all()
    t = torch.from_numpy(y).float()  # (a library's conversion, of numbers that it does not saturate)
    keep = t.abs() < 448
    same = R.code(t.double().numpy()) == t.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert (same | ~keep.numpy() | (R.code(t.double().numpy()) == 0)).all()
    assert [R.scale_exponent(x) for x in (0.0, 1.0, 1.01, 2.0, 2.0**-60, 2.0**100)] == [-40, -8, -7, -7, -40, 40]


def append(lib, **kw):
    a = dict(k=A, kb=1024, kt=512, kh=128, v=A, vb=1024, vt=512, vh=128, dtype=1, B=2, T=2, H=4, D=128, cache=A, pages=9, page=16,
             table=A, width=4, start=A, new=None, cos=A, sin=A, len=64, pairs=64, inter=0, pos=None, kv=None, vv=None)
    a.update(kw)
    return lib.spec_kv8_append(*a.values(), None)


@pytest.mark.parametrize("kw,status", S.SHARED + [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(k=A + 1), INVALID), (dict(kb=-1), INVALID), (dict(vh=-1), INVALID),
    (dict(kv=A + 2), INVALID), (dict(vv=A + 4), INVALID), (dict(T=1 << 30, H=16), INVALID), (dict(T=1 << 30, H=4, B=1 << 20), INVALID)])
def test_append_refusals(lib, kw, status):
    assert append(lib, **kw) == status


def attend(lib, **kw):
    a = dict(q=A, qb=4096, qt=2048, qh=128, dtype=1, B=2, T=2, Hq=16, H=4, D=128, cache=A, pages=9, page=16, table=A, width=4,
             start=A, new=None, parent=None, scale=0.1, cos=A, sin=A, len=64, pairs=64, inter=0, pos=None, out=A, ws=A, n=1 << 40)
    a.update(kw)
    return lib.spec_kv8_attention(*a.values(), None)


@pytest.mark.parametrize("kw,status", S.SHARED + [
    (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(q=A + 1), INVALID), (dict(out=A + 8), INVALID), (dict(Hq=15), INVALID),
    (dict(Hq=0), INVALID), (dict(qt=-1), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(T=1025, parent=A), INVALID), (dict(T=1 << 28), INVALID), (dict(ws=None), WORKSPACE), (dict(ws=A + 8), WORKSPACE),
    (dict(n=100), WORKSPACE)])
def test_attention_refusals(lib, kw, status):
    assert attend(lib, **kw) == status


@pytest.mark.parametrize("D,Hq,T", [(64, 4, 1), (64, 16, 40), (128, 16, 9), (256, 8, 1), (256, 16, 40)])
def test_attention_capacity_limit(lib, D, Hq, T):
    most = (1 << 31) - 128
    for page in (16, 128):
        call = dict(D=D, Hq=Hq, T=T, pairs=D // 2, page=page, ws=None)
        assert attend(lib, width=most // page, **call) == WORKSPACE
        assert attend(lib, width=most // page + 1, **call) == INVALID


def test_attention_workspace_size(lib):
    size = sv.spec_kv8_attention_workspace_size
    assert size(0, 1, 8, 8, 128) == size(1, 0, 8, 8, 128) == size(1, 1, 8, 3, 128) == size(1, 1, 8, 8, 96) == 0
    # two partial results per thread block: 16 rows of D floats, a maximum and a sum each; and three bytes a number of the queries
    assert size(1, 1, 8, 8, 128) >= 152 * 2 * 16 * (128 + 2) * 4 + 8 * 16 * 3 * 128
    assert size(500, 1, 64, 8, 128) - size(1, 1, 64, 8, 128) >= 499 * 8 * 16 * 3 * 128
    assert size(4, 9, 32, 8, 128) % 256 == 0


def read(lib, **kw):
    a = dict(cache=A, pages=9, page=16, B=2, T=5, H=4, D=128, table=A, width=4, start=A, lens=None, slots=None, dtype=1, k=A, v=A)
    a.update(kw)
    return lib.spec_kv8_read(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=0), UNSUPPORTED), (dict(dtype=3), UNSUPPORTED), (dict(D=96), UNSUPPORTED), (dict(page=24), UNSUPPORTED),
    (dict(page=2048), UNSUPPORTED), (dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(pages=-1), INVALID),
    (dict(width=-1), INVALID), (dict(width=1 << 27), INVALID), (dict(cache=A + 8), INVALID), (dict(cache=None), INVALID),
    (dict(table=None), INVALID), (dict(start=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(k=A + 2), INVALID),
    (dict(v=A + 8), INVALID), (dict(T=(1 << 31) - 1, H=16), INVALID), (dict(T=1 << 28, B=64), INVALID),
    (dict(B=0, cache=None, start=None), OK), (dict(T=0), OK)])
def test_read_refusals(lib, kw, status):
    assert read(lib, **kw) == status


def test_bindings_refuse_what_they_cannot_take(lib):
    h = torch.zeros((1, 1, 2, 64), dtype=torch.bfloat16)
    cache = torch.zeros((1, 2, 16 * 129), dtype=torch.uint8)
    i = torch.zeros((1, 1), dtype=torch.int32)
    for call in (lambda: sv.spec_kv8_append(h, h, cache, i, i[0]), lambda: sv.spec_kv8_attention(h, cache, i, i[0]),
                 lambda: sv.spec_kv8_read(cache, i, i[0], 3)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
