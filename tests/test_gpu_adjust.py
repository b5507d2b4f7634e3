"""spec_logit_adjust against its formula in 64 bits.

Tolerance: five fp32 operations (2^-24 of a term's magnitude each; 8 allowed), then one rounding to the
output's type (half a step of it)."""
import numpy as np
import pytest
import torch

import speculative_decoding_verify_spec_gb300 as sv
from tests import serve_util as U

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def inputs(B, R, V, dtype, n=40, tree=False, bias=5, grammar=True, seed=0):
    g = torch.Generator().manual_seed(seed)
    d = dict(logits=(torch.randn((B, R, V), generator=g) * 4).to(DT[dtype]))
    tok = lambda *s: ((torch.rand(s, generator=g) ** 2) * V).to(torch.int32)  # noqa: E731
    if n:
        d["history"], d["lengths"] = tok(B, n), torch.randint(0, n + 1, (B,), generator=g, dtype=torch.int32)
        d["prompt_lengths"] = torch.randint(0, n, (B,), generator=g, dtype=torch.int32)
    if tree:
        d["parent"] = torch.tensor([-1] + [int(torch.randint(max(0, i - 3), i, (1,), generator=g)) for i in range(1, R)], dtype=torch.int32)
    d["draft_tokens"] = tok(B, R if tree else R - 1)
    d["repetition"] = 0.7 + torch.rand(B, generator=g)
    d["frequency"], d["presence"] = torch.rand(B, generator=g), torch.randn(B, generator=g)
    if bias:
        d["bias_tokens"], d["bias_values"] = tok(B, bias), torch.randn((B, bias), generator=g) * 5
    if grammar:
        d["allowed"] = torch.randint(-2**31, 2**31 - 1, (B, R, (V + 31) // 32), generator=g, dtype=torch.int64).to(torch.int32)
    return d


def call(d, **kw):
    return sv.spec_logit_adjust(**{k: v.to(DEV) for k, v in d.items()}, **kw)


def check(d, got):
    want, mag = U.adjust(**d)
    x = got.double().cpu().numpy()
    with np.errstate(invalid="ignore"):
        tol = 8 * 2.0**-24 * mag + (np.abs(want) * U.half_step(d["logits"].dtype) if d["logits"].dtype != torch.float32 else 0)
        same = (x == want) | (np.isnan(x) & np.isnan(want))
        assert (same | (np.abs(x - want) <= tol)).all()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("B,R,V,n", [(1, 1, 1, 1), (2, 3, 7, 40), (1, 5, 1000, 200), (3, 4, 1023, 65), (2, 2, 4096, 33),
                                     (5, 9, 4099, 500), (2, 3, 12345, 4001), (130, 2, 9001, 64)])
def test_chain(dtype, B, R, V, n):
    d = inputs(B, R, V, dtype, n)
    check(d, call(d))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("B,R,V", [(1, 1, 100), (2, 17, 515), (3, 64, 5000), (1, 200, 77)])
def test_tree(dtype, B, R, V):
    d = inputs(B, R, V, dtype, tree=True)
    check(d, call(d))
    d["parent"][R // 2] = R + 3  # a malformed entry ends the path
    check(d, call(d))


@pytest.mark.parametrize("drop", [["history", "lengths", "prompt_lengths"], ["prompt_lengths"], ["draft_tokens"], ["repetition"],
                                  ["frequency", "presence"], ["bias_tokens", "bias_values"], ["allowed"],
                                  ["history", "lengths", "prompt_lengths", "draft_tokens", "bias_tokens", "bias_values", "allowed"]])
def test_each_part_may_be_left_out(drop):
    d = inputs(2, 4, 3001, "bf16")
    for k in drop:
        del d[k]
    check(d, call(d))


def test_repeated_drafts_bias_duplicates_and_tokens_outside():
    d = inputs(2, 6, 50, "fp32", n=30, bias=20)
    d["draft_tokens"][:] = 3
    d["draft_tokens"][0, 1] = -1
    d["draft_tokens"][1, 2] = 50
    d["history"][0, :10] = torch.tensor([-1, 50, 2**31 - 1, -2**31, 3, 3, 49, 0, 0, 7], dtype=torch.int32)
    d["bias_tokens"][:, ::3] = 11  # the last of them counts
    d["bias_tokens"][:, 1] = -5
    d["bias_tokens"][:, 2] = 1 << 30
    check(d, call(d))
    d["lengths"][:] = torch.tensor([-4, 1000], dtype=torch.int32)  # clamped
    d["prompt_lengths"][:] = torch.tensor([5, -1], dtype=torch.int32)
    check(d, call(d))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_infinities_nan_and_empty_rows(dtype):
    d = inputs(2, 3, 700, dtype)
    d["logits"][0, 0, ::7] = float("-inf")
    d["logits"][0, 1, ::5] = float("inf")
    d["logits"][1, 0, ::3] = float("nan")
    d["logits"][1, 1, ::4] = torch.finfo(DT[dtype]).min
    d["allowed"][1, 2] = 0  # nothing allowed
    d["allowed"][0, 0] = -1  # all
    got = call(d)
    check(d, got)
    assert torch.isneginf(got[1, 2]).all()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("V", [1000, 1001, 5003])
def test_strides_alignment_and_in_place(dtype, V):
    d = inputs(3, 4, V, dtype)
    dev = {k: v.to(DEV) for k, v in d.items()}
    want = sv.spec_logit_adjust(**dev)
    for pad_in, off_in, pad_out, off_out in ((8, 0, 8, 0), (3, 1, 3, 1), (0, 1, 0, 2), (5, 3, 0, 0)):
        a = torch.empty(3 * (4 * (V + pad_in) + 7) + off_in, dtype=DT[dtype], device=DEV)
        src = a[off_in:].as_strided((3, 4, V), (4 * (V + pad_in) + 7, V + pad_in, 1))
        src.copy_(dev["logits"])
        o = torch.full((3 * (4 * (V + pad_out) + 5) + off_out,), 123.0, dtype=DT[dtype], device=DEV)
        dst = o[off_out:].as_strided((3, 4, V), (4 * (V + pad_out) + 5, V + pad_out, 1))
        keep = o.clone()
        keep[off_out:].as_strided(dst.shape, dst.stride()).copy_(want)
        sv.spec_logit_adjust(**{**dev, "logits": src}, out=dst)
        assert torch.equal(o, keep)  # and nothing around the rows
        sv.spec_logit_adjust(**{**dev, "logits": src}, out=src)  # in place
        assert torch.equal(src, want)
    one = dev["logits"][:1, :1].expand(3, 4, V)  # broadcast rows
    assert torch.equal(sv.spec_logit_adjust(**{**dev, "logits": one}), sv.spec_logit_adjust(**{**dev, "logits": one.contiguous()}))


def test_graph_capture_and_other_streams():
    d = {k: v.to(DEV) for k, v in inputs(4, 5, 4003, "bf16").items()}
    want = sv.spec_logit_adjust(**d)
    out = torch.empty_like(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        sv.spec_logit_adjust(**d, out=out)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.spec_logit_adjust(**d, out=out)
    out.zero_()
    graph.replay()
    assert torch.equal(out, want)


def test_empty_and_refused():
    d = {k: v.to(DEV) for k, v in inputs(2, 3, 64, "bf16").items()}
    assert sv.spec_logit_adjust(d["logits"][:0]).shape == (0, 3, 64)
    assert sv.spec_logit_adjust(d["logits"][:, :0]).shape == (2, 0, 64)
    with pytest.raises(TypeError):
        sv.spec_logit_adjust(d["logits"].half())
    for bad in (dict(history=d["history"]), dict(allowed=d["allowed"][:, :, :1]), dict(repetition=d["repetition"][:1]),
                dict(draft_tokens=d["draft_tokens"][:, :1]), dict(bias_tokens=d["bias_tokens"]), dict(out=d["logits"].float()),
                dict(parent=torch.zeros(3, dtype=torch.int32, device=DEV)), dict(lengths=1, history=d["history"].long())):
        with pytest.raises((ValueError, AttributeError)):
            sv.spec_logit_adjust(d["logits"], **bad)
    with pytest.raises(sv.SpecVerifyError, match="status 1"):
        sv.spec_logit_adjust(d["logits"], out=torch.empty((1, 1, 64), dtype=torch.bfloat16, device=DEV).expand(2, 3, 64))
