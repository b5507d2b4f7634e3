"""Python entry points of the operators around the verification step (``include/spec_serve.h``).

``spec_logit_adjust`` applies penalties, biases and grammar masks to the verified rows' logits;
``spec_kv_append`` and ``spec_kv_attention`` keep and read a paged key/value cache held in 4 bits,
``spec_kv8_append``, ``spec_kv8_read`` and ``spec_kv8_attention`` one held in 8 bits.
As in ``binding``, these only marshal: they check placement, type and shape, take strides and
the current stream from PyTorch and call the C entry of the same name.
"""
from __future__ import annotations

import ctypes
import functools
import math

import torch

from . import binding
from .binding import _check, _dtype_code, _ints, _logits3, _stream

KV_BF16, KV_FP16 = 1, 2
_ready = None


def _library() -> ctypes.CDLL:
    global _ready
    if _ready is None:
        lib = binding.load_library()
        P, i64, i32, f32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        lib.spec_logit_adjust.argtypes = [P, i64, i64, P, i64, i64, i32, i32, i32, i32, P, i64, P, P, P, P, P, P, P, P,
                                          P, i32, P, P]
        lib.spec_logit_adjust.restype = i32
        lib.spec_kv_page_bytes.argtypes = [i32, i32]
        lib.spec_kv_page_bytes.restype = sz
        lib.spec_kv_code_offset.argtypes = [i32] * 5
        lib.spec_kv_code_offset.restype = i64
        lib.spec_kv_append.argtypes = [P, i64, i64, i64, P, i64, i64, i64, i32, i32, i32, i32, i32, P, i32, i32, P, i32,
                                       P, P, P, P, i32, i32, i32, P, P, P, P]
        lib.spec_kv_append.restype = i32
        lib.spec_kv_attention_workspace_size.argtypes = [i32] * 5
        lib.spec_kv_attention_workspace_size.restype = sz
        lib.spec_kv_attention.argtypes = [P, i64, i64, i64, i32, i32, i32, i32, i32, i32, P, i32, i32, P, i32, P, P, P,
                                          f32, P, P, i32, i32, i32, P, P, P, sz, P]
        lib.spec_kv_attention.restype = i32
        lib.spec_kv8_page_bytes.argtypes = [i32, i32]
        lib.spec_kv8_page_bytes.restype = sz
        lib.spec_kv8_code_offset.argtypes = [i32] * 5
        lib.spec_kv8_code_offset.restype = i64
        lib.spec_kv8_append.argtypes = lib.spec_kv_append.argtypes
        lib.spec_kv8_append.restype = i32
        lib.spec_kv8_read.argtypes = [P, i32, i32, i32, i32, i32, i32, P, i32, P, P, P, i32, P, P, P]
        lib.spec_kv8_read.restype = i32
        lib.spec_kv8_attention_workspace_size.argtypes = [i32] * 5
        lib.spec_kv8_attention_workspace_size.restype = sz
        lib.spec_kv8_attention.argtypes = lib.spec_kv_attention.argtypes
        lib.spec_kv8_attention.restype = i32
        lib.spec_kv_lose_unit.argtypes = [i32]
        lib.spec_kv_lose_unit.restype = i32
        _ready = lib
    return _ready


# The checks below take their common case first: a call's host time is what a small step waits for.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _current(dev) -> int:
    """The current stream's handle on dev."""
    return _raw_stream(dev.index) if _raw_stream is not None and dev.index is not None else _stream(dev)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _like(t):
    """A new contiguous tensor of t's shape and type."""
    return torch.empty_like(t, memory_format=torch.contiguous_format)


def _int32(t, name, shape, dev):
    """t, an int32 tensor of that shape on dev (or None), contiguous."""
    if t is None or (t.dtype is torch.int32 and t.shape == shape and t.get_device() == dev.index and t.is_contiguous()):
        return t
    return _ints(t, name, shape, dev)


def _floats(t, name, shape, dev):
    if t is None or (t.dtype is torch.float32 and t.shape == shape and t.get_device() == dev.index and t.is_contiguous()):
        return t
    if t.dtype != torch.float32 or t.device != dev or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be float32 of shape {tuple(shape)} on {dev}")
    return t.contiguous()


def spec_logit_adjust(logits: torch.Tensor, *, history=None, lengths=None, prompt_lengths=None, draft_tokens=None,
                      parent=None, repetition=None, frequency=None, presence=None, bias_tokens=None, bias_values=None,
                      allowed=None, out=None) -> torch.Tensor:
    """Penalties, biases and grammar masks on logits [B, rows, V] (bf16 or fp32); returns `out`, a new
    contiguous tensor unless given (`out=logits` works in place).

    The context of row i is the history ([B, n] int32 with `lengths` [B], the first `prompt_lengths`
    [B] of them the prompt) and the drafts before it: `draft_tokens` [B, rows - 1] for a chain, or the path
    to node i of the tree `parent` [rows] with `draft_tokens` [B, rows] (node 0, the root, is the history's
    last token).  Tokens in the context have their logit divided (if positive) or multiplied by `repetition`
    [B]; those in its output part lose `frequency` [B] per occurrence and `presence` [B] once; then
    `bias_values` [B, n] fp32 are added to `bias_tokens` [B, n] (the last entry of a token counts, tokens outside the
    vocabulary are unused); last, tokens whose bit in `allowed` [B, rows, ceil(V / 32)] int32 is clear become -inf."""
    lib = _library()
    sb, sr = _logits3(logits, "logits")
    B, R, V = logits.shape
    dt, dev, row = _dtype_code(logits), logits.device, (B,)
    if out is None:
        out = _like(logits)
        ob, orow, _ = out.stride()
    elif out.device != dev or out.dtype != logits.dtype or tuple(out.shape) != (B, R, V):
        raise ValueError(f"out must be {logits.dtype} of shape {(B, R, V)} on {dev}")
    else:
        ob, orow = _logits3(out, "out")
    n = 0
    if history is not None:
        if history.dim() != 2 or lengths is None:
            raise ValueError("history must be [B, n], with lengths [B]")
        n = history.shape[1]
        history = _int32(history, "history", (B, n), dev)
        lengths = _int32(lengths, "lengths", row, dev)
        prompt_lengths = _int32(prompt_lengths, "prompt_lengths", row, dev)
    if parent is not None:
        if draft_tokens is None:
            raise ValueError("a tree (parent) needs draft_tokens [B, rows]")
        parent = _int32(parent, "parent", (R,), dev)
    if draft_tokens is not None:
        draft_tokens = _int32(draft_tokens, "draft_tokens", (B, R if parent is not None else max(R - 1, 0)), dev)
    k = 0
    if (bias_tokens is None) != (bias_values is None):
        raise ValueError("bias_tokens and bias_values belong together")
    if bias_tokens is not None:
        k = bias_tokens.shape[1] if bias_tokens.dim() == 2 else -1
        bias_tokens = _int32(bias_tokens, "bias_tokens", (B, k), dev)
        bias_values = _floats(bias_values, "bias_values", (B, k), dev)
    repetition = _floats(repetition, "repetition", row, dev)
    frequency = _floats(frequency, "frequency", row, dev)
    presence = _floats(presence, "presence", row, dev)
    allowed = _int32(allowed, "allowed", (B, R, (V + 31) // 32), dev)
    st = lib.spec_logit_adjust(logits.data_ptr(), sb, sr, out.data_ptr(), ob, orow, dt, B, R, V, _ptr(history), n,
                               _ptr(lengths), _ptr(prompt_lengths), _ptr(draft_tokens), _ptr(parent), _ptr(repetition),
                               _ptr(frequency), _ptr(presence), _ptr(bias_tokens), _ptr(bias_values), k, _ptr(allowed),
                               _current(dev))
    _check(st, "spec_logit_adjust")
    return out


def spec_kv_page_bytes(page_size: int, head_dim: int) -> int:
    """Bytes of one page and head of the 4-bit cache (0 if the sizes are not supported)."""
    return int(_library().spec_kv_page_bytes(page_size, head_dim))


def _kv_dtype(t: torch.Tensor, name: str) -> int:
    if t.dtype == torch.bfloat16:
        return KV_BF16
    if t.dtype == torch.float16:
        return KV_FP16
    raise TypeError(f"{name} must be bfloat16 or float16, got {t.dtype}")


def _heads4(t: torch.Tensor, name: str):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    st = t.stride()
    if len(st) != 4 or (st[3] != 1 and t.shape[3] > 1):
        raise ValueError(f"{name} must be [B, T, heads, head_dim] with a contiguous last axis")
    return st


def _cache(cache, page_table, start, new_lens, B, heads, D, dev, slot_bytes=0):
    """(num_pages, page_size, checked page_table, its width, start, new_lens) of a checked cache; slot_bytes: of a token and
    head, unless it is the 4-bit cache."""
    cs = cache.shape
    if cache.dtype is not torch.uint8 or len(cs) != 3 or cache.get_device() != dev.index or not cache.is_contiguous():
        raise ValueError(f"cache must be a contiguous uint8 tensor [pages, kv_heads, page bytes] on {dev}")
    page, rest = divmod(cs[2], slot_bytes or D + 8)
    if (heads is not None and cs[1] != heads) or rest:
        raise ValueError(f"cache of shape {tuple(cs)} does not hold {heads} heads of {D} dimensions")
    ps = page_table.shape
    if len(ps) != 2:
        raise ValueError("page_table must be [B, pages per sequence]")
    width, row = ps[1], (B,)
    return (cs[0], page, _int32(page_table, "page_table", (B, width), dev), width, _int32(start, "start", row, dev),
            _int32(new_lens, "new_lens", row, dev))


def _rotation(cos, sin, positions, B, T, dev):
    if cos is None and sin is None:
        return None, None, 0, 0, None
    if cos is None or sin is None:
        raise ValueError("cos and sin belong together")
    shape = cos.shape
    if len(shape) != 2:
        raise ValueError("cos must be [positions, pairs]")
    return (_floats(cos, "cos", shape, dev), _floats(sin, "sin", shape, dev), shape[0], shape[1],
            _int32(positions, "positions", (B, T), dev))


def spec_kv_append(k: torch.Tensor, v: torch.Tensor, cache: torch.Tensor, page_table: torch.Tensor, start: torch.Tensor,
                   *, new_lens=None, cos=None, sin=None, positions=None, interleaved: bool = False,
                   return_values: bool = False, k_values=None, v_values=None):
    """Writes the new tokens' keys (rotated) and values [B, T, kv_heads, head_dim] into the 4-bit `cache`
    [pages, kv_heads, spec_kv_page_bytes(page_size, head_dim)] uint8, as tokens start[b] .. of sequence b
    (`new_lens` [B] of them, all T if None), in the pages that `page_table` [B, n] names.

    cos, sin [positions, pairs] fp32 turn the first 2 * pairs dimensions by the angles of the tokens' positions
    (`positions` [B, T], else start[b] + t).  With `return_values`, or `k_values` and `v_values` given, returns what the
    cache now holds for the new tokens, in the inputs' type (0 from new_lens[b] on; for a token dropped at the table's end or at a
    page out of range, what it would have been held as); else None."""
    lib = _library()
    ks, dt, dev, shape = _heads4(k, "k"), _kv_dtype(k, "k"), k.device, k.shape
    vs = _heads4(v, "v")
    if v.shape != shape or v.dtype != k.dtype or v.device != dev:
        raise ValueError("v must have k's shape, type and device")
    B, T, H, D = shape
    pages, page, page_table, width, start, new_lens = _cache(cache, page_table, start, new_lens, B, H, D, dev)
    cos, sin, length, pairs, positions = _rotation(cos, sin, positions, B, T, dev)
    for name, t in (("k_values", k_values), ("v_values", v_values)):
        if t is not None and (t.shape != shape or t.dtype != k.dtype or t.device != dev or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous tensor like k")
    if return_values:
        k_values = _like(k) if k_values is None else k_values
        v_values = _like(k) if v_values is None else v_values
    st = lib.spec_kv_append(k.data_ptr(), ks[0], ks[1], ks[2], v.data_ptr(), vs[0], vs[1], vs[2], dt, B, T, H, D, cache.data_ptr(), pages, page,
                            page_table.data_ptr(), width, start.data_ptr(), _ptr(new_lens), _ptr(cos), _ptr(sin), length,
                            pairs, int(interleaved), _ptr(positions), _ptr(k_values), _ptr(v_values), _current(dev))
    _check(st, "spec_kv_append")
    return None if k_values is None and v_values is None else (k_values, v_values)


@functools.lru_cache(maxsize=1024)
def spec_kv_attention_workspace_size(B: int, T: int, heads: int, kv_heads: int, head_dim: int) -> int:
    """Bytes of workspace that spec_kv_attention needs for these sizes."""
    return int(_library().spec_kv_attention_workspace_size(B, T, heads, kv_heads, head_dim))


def spec_kv_attention(q: torch.Tensor, cache: torch.Tensor, page_table: torch.Tensor, start: torch.Tensor, *,
                      new_lens=None, parent=None, scale=None, cos=None, sin=None, positions=None,
                      interleaved: bool = False, workspace=None, out=None) -> torch.Tensor:
    """Attention of the step's new tokens' queries [B, T, heads, head_dim] over the 4-bit cache, which holds
    the new tokens already (see spec_kv_append: same cache, page_table, start, new_lens and rotation).

    Token t sees the tokens before start[b], and of the new ones 0 .. t (a chain), or its ancestors and itself
    if `parent` [T] gives a tree.  scale defaults to head_dim ** -0.5.  Returns [B, T, heads, head_dim].

    The first int32 of `workspace` (spec_kv_attention_workspace_size bytes; one of the call's own unless given) is the call's status
    once the stream has completed: 0, or 4 if a bounded wait on the device gave up; the result is then NaN throughout."""
    lib = _library()
    qs, dt, dev = _heads4(q, "q"), _kv_dtype(q, "q"), q.device
    B, T, Hq, D = q.shape
    H = cache.shape[1] if cache.dim() == 3 else 0
    if H < 1 or Hq % H:
        raise ValueError(f"{Hq} query heads do not share the cache's heads (shape {tuple(cache.shape)}) evenly")
    pages, page, page_table, width, start, new_lens = _cache(cache, page_table, start, new_lens, B, None, D, dev)
    cos, sin, length, pairs, positions = _rotation(cos, sin, positions, B, T, dev)
    if parent is not None:
        parent = _int32(parent, "parent", (T,), dev)
    if out is None:
        out = _like(q)
    elif out.shape != q.shape or out.dtype != q.dtype or out.device != dev or not out.is_contiguous():
        raise ValueError("out must be a contiguous tensor like q")
    n = spec_kv_attention_workspace_size(B, T, Hq, H, D)
    if workspace is None:
        workspace = torch.empty(max(n, 16), dtype=torch.uint8, device=dev)
    else:
        if workspace.device != dev or not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous tensor on {dev}")
        n = workspace.numel() * workspace.element_size()
    st = lib.spec_kv_attention(q.data_ptr(), qs[0], qs[1], qs[2], dt, B, T, Hq, H, D, cache.data_ptr(), pages, page, page_table.data_ptr(),
                               width, start.data_ptr(), _ptr(new_lens), _ptr(parent),
                               1.0 / math.sqrt(D) if scale is None else float(scale), _ptr(cos), _ptr(sin), length, pairs,
                               int(interleaved), _ptr(positions), out.data_ptr(), workspace.data_ptr(), n, _current(dev))
    _check(st, "spec_kv_attention")
    return out


def spec_kv8_page_bytes(page_size: int, head_dim: int) -> int:
    """Bytes of one page and head of the 8-bit cache (0 if the sizes are not supported)."""
    return int(_library().spec_kv8_page_bytes(page_size, head_dim))


def spec_kv8_append(k: torch.Tensor, v: torch.Tensor, cache: torch.Tensor, page_table: torch.Tensor, start: torch.Tensor,
                    *, new_lens=None, cos=None, sin=None, positions=None, interleaved: bool = False,
                    return_values: bool = False, k_values=None, v_values=None):
    """Writes the new tokens' keys (rotated) and values [B, T, kv_heads, head_dim] into the 8-bit `cache`
    [pages, kv_heads, spec_kv8_page_bytes(page_size, head_dim)] uint8; arguments and result as for spec_kv_append.

    A number is held as a float of 8 bits (3 of mantissa) times a scale, a power of two, which 16 neighbouring slots of a head share.
    Where a new token is louder than the tokens that its block of 16 holds already, these are rounded to the larger scale (exact but for
    numbers 2^14 times smaller than the largest)."""
    lib = _library()
    ks, dt, dev, shape = _heads4(k, "k"), _kv_dtype(k, "k"), k.device, k.shape
    vs = _heads4(v, "v")
    if v.shape != shape or v.dtype != k.dtype or v.device != dev:
        raise ValueError("v must have k's shape, type and device")
    B, T, H, D = shape
    pages, page, page_table, width, start, new_lens = _cache(cache, page_table, start, new_lens, B, H, D, dev, 2 * D + 1)
    cos, sin, length, pairs, positions = _rotation(cos, sin, positions, B, T, dev)
    for name, t in (("k_values", k_values), ("v_values", v_values)):
        if t is not None and (t.shape != shape or t.dtype != k.dtype or t.device != dev or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous tensor like k")
    if return_values:
        k_values = _like(k) if k_values is None else k_values
        v_values = _like(k) if v_values is None else v_values
    st = lib.spec_kv8_append(k.data_ptr(), ks[0], ks[1], ks[2], v.data_ptr(), vs[0], vs[1], vs[2], dt, B, T, H, D, cache.data_ptr(), pages, page,
                             page_table.data_ptr(), width, start.data_ptr(), _ptr(new_lens), _ptr(cos), _ptr(sin), length,
                             pairs, int(interleaved), _ptr(positions), _ptr(k_values), _ptr(v_values), _current(dev))
    _check(st, "spec_kv8_append")
    return None if k_values is None and v_values is None else (k_values, v_values)


def _head_dim8(page_bytes: int) -> int:
    """The head dimension of an 8-bit cache with such pages (no two have a page size with the same bytes)."""
    for D in (64, 128, 256):
        page, rest = divmod(page_bytes, 2 * D + 1)
        if rest == 0 and page % 16 == 0 and 16 <= page <= 1024:
            return D
    raise ValueError(f"pages of {page_bytes} bytes are not those of an 8-bit cache (see spec_kv8_page_bytes)")


def spec_kv8_read(cache: torch.Tensor, page_table: torch.Tensor, start: torch.Tensor, T: int, *, lens=None, slots=None,
                  dtype: torch.dtype = torch.bfloat16, k=None, v=None):
    """Tokens of the 8-bit cache back in 16 bits: (keys, values) [B, T, kv_heads, head_dim], new unless `k` and `v` are given.

    Row t of sequence b is its token start[b] + t, or slots[b, t] if `slots` [B, T] int32 is given (a tree's accepted path, to be
    appended again behind the context); `lens` [B] of the rows are read, all T if None.  Rows from lens[b] on, tokens outside the
    page table and pages out of range are 0.  Keys come as they are held, rotated."""
    lib = _library()
    if not cache.is_cuda or cache.dim() != 3:
        raise ValueError("cache must be a CUDA tensor [pages, kv_heads, page bytes]")
    dev, H, D, B, T = cache.device, cache.shape[1], _head_dim8(cache.shape[2]), page_table.shape[0], int(T)
    if T < 0:
        raise ValueError(f"T must not be negative, got {T}")
    pages, page, page_table, width, start, lens = _cache(cache, page_table, start, lens, B, H, D, dev, 2 * D + 1)
    slots = _int32(slots, "slots", (B, T), dev)
    if k is None:
        k = torch.empty((B, T, H, D), dtype=dtype, device=dev)
    if v is None:
        v = torch.empty((B, T, H, D), dtype=k.dtype, device=dev)
    for name, t in (("k", k), ("v", v)):
        if t.shape != (B, T, H, D) or t.dtype != k.dtype or t.device != dev or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous tensor of {k.dtype} and shape {(B, T, H, D)} on {dev}")
    st = lib.spec_kv8_read(cache.data_ptr(), pages, page, B, T, H, D, page_table.data_ptr(), width, start.data_ptr(), _ptr(lens), _ptr(slots),
                           _kv_dtype(k, "k"), k.data_ptr(), v.data_ptr(), _current(dev))
    _check(st, "spec_kv8_read")
    return k, v


@functools.lru_cache(maxsize=1024)
def spec_kv8_attention_workspace_size(B: int, T: int, heads: int, kv_heads: int, head_dim: int) -> int:
    """Bytes of workspace that spec_kv8_attention needs for these sizes."""
    return int(_library().spec_kv8_attention_workspace_size(B, T, heads, kv_heads, head_dim))


def spec_kv8_attention(q: torch.Tensor, cache: torch.Tensor, page_table: torch.Tensor, start: torch.Tensor, *,
                       new_lens=None, parent=None, scale=None, cos=None, sin=None, positions=None,
                       interleaved: bool = False, workspace=None, out=None) -> torch.Tensor:
    """Attention of the step's new tokens' queries [B, T, heads, head_dim] over the 8-bit cache, which holds the new tokens
    already (see spec_kv8_append); arguments, result and the workspace's status word as for spec_kv_attention."""
    lib = _library()
    qs, dt, dev = _heads4(q, "q"), _kv_dtype(q, "q"), q.device
    B, T, Hq, D = q.shape
    H = cache.shape[1] if cache.dim() == 3 else 0
    if H < 1 or Hq % H:
        raise ValueError(f"{Hq} query heads do not share the cache's heads (shape {tuple(cache.shape)}) evenly")
    pages, page, page_table, width, start, new_lens = _cache(cache, page_table, start, new_lens, B, None, D, dev, 2 * D + 1)
    cos, sin, length, pairs, positions = _rotation(cos, sin, positions, B, T, dev)
    if parent is not None:
        parent = _int32(parent, "parent", (T,), dev)
    if out is None:
        out = _like(q)
    elif out.shape != q.shape or out.dtype != q.dtype or out.device != dev or not out.is_contiguous():
        raise ValueError("out must be a contiguous tensor like q")
    n = spec_kv8_attention_workspace_size(B, T, Hq, H, D)
    if workspace is None:
        workspace = torch.empty(max(n, 16), dtype=torch.uint8, device=dev)
    else:
        if workspace.device != dev or not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous tensor on {dev}")
        n = workspace.numel() * workspace.element_size()
    st = lib.spec_kv8_attention(q.data_ptr(), qs[0], qs[1], qs[2], dt, B, T, Hq, H, D, cache.data_ptr(), pages, page, page_table.data_ptr(),
                                width, start.data_ptr(), _ptr(new_lens), _ptr(parent),
                                1.0 / math.sqrt(D) if scale is None else float(scale), _ptr(cos), _ptr(sin), length, pairs,
                                int(interleaved), _ptr(positions), out.data_ptr(), workspace.data_ptr(), n, _current(dev))
    _check(st, "spec_kv8_attention")
    return out


def lose_unit(unit: int) -> int:
    """Test hook of the bounds-checked build (see spec_kv_lose_unit); returns the status."""
    return int(_library().spec_kv_lose_unit(unit))
