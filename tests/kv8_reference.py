"""The operators of the 8-bit paged cache in 64 bits, and what bounds the attention's error, element by element.

Errors of the attention, with s_j and s'_j the scales of token j's key and value, c'_j its value's codes:
- a query is held in two parts of 8 bits each where it is bf16 and not rotated, in three else, its row's largest number in 2^7 .. 2^8.
  Each part keeps 4 significant bits of what the parts before it left (half a step is 2^-4 of it), and bf16 has 8: what is lost is at most
  2^-12 of a number (0 in the first case) and half of the smallest step, 2^-10, or 2^-17 of the row's largest number;
- a weight w_j = p_j s'_j is held in two such parts for bf16 outputs, in three for fp16 ones, the largest of a tile of 128 tokens in
  2^7.5 .. 2^8.5: off by 2^-8 or 2^-12 of itself, and by 2^-10 / 2^7.5 of the tile's largest.  These roundings are independent and at most half a
  step each, uniform or narrower within it (a deviation of 1 / sqrt(3)): the error of a sum of them is within its linear bound, and within
  six deviations, 3.5 times the root of the sum of their squares;
- a score is an fp32 sum of products, 2^-20 of the sum of their sizes (an exact product needs 8 bits; sums of D and of three parts, each step
  2^-23 or less); the shift by log2 s' and the maximum, and the exponential: 2^-21 (1 + |log2 s'|);
- the tiles' sums, of 128 products, and theirs, in fp32: 2^-23 each of the sum of sizes, 128 + tiles of them at most, in which the random
  directions are not counted on;
- the output is rounded to its type."""
import math

import numpy as np
import torch

from tests import serve_util as U

TILE = 128
NUMBERS = np.array([(-1.0) ** (n >> 7) * ((n & 7) * 2.0**-9 if n & 120 == 0 else (8 + (n & 7)) * 2.0 ** ((n >> 3 & 15) - 10)) for n in range(256)])
NUMBERS[[127, 255]] = np.nan


def place(D, slot, d):
    """Byte of a code among the keys' or the values' codes of a page and head."""
    return slot // 8 * 8 * D + d // 16 * 128 + slot % 8 * 16 + d % 16


def code(y):
    """Codes nearest to y (float64), ties to the even one, 448 at most, zero as +0."""
    m = np.minimum(np.abs(y), 448.0)
    e = np.maximum(np.frexp(m)[1] - 1, -6)
    n = np.rint(np.ldexp(m, 3 - e)).astype(int)
    c = np.where(n >= 8, (e + 6) * 8 + n, n)
    return np.where((y < 0) & (c > 0), c + 128, c).astype(np.uint8)


def scale_exponent(largest):
    """Of the least scale that the rule gives for a largest magnitude."""
    if largest == 0:
        return -40
    m, e = math.frexp(largest)
    return min(max((e - 1 if m == 0.5 else e) - 8, -40), 40)


def word(cache, page, D, pg, h, slot, values):
    at = 2 * page * D + slot // 16 * 16 + 4 * values
    return int(cache[pg, h, at:at + 4].copy().view(np.uint32)[0])


def old_exponent(w):
    return min(max((w >> 23 & 255) - 127, -40), 40)


def append(cache, table, k, v, start, new, page):
    """(the cache's bytes, [held keys, held values] [B, T, H, D]) after appending rotated keys k and values v [B, T, H, D] float64."""
    want = cache.copy()
    pages, H, _ = want.shape
    B, T, _, D = k.shape
    cap = table.shape[1] * page
    held = [np.zeros(k.shape), np.zeros(k.shape)]
    dims = np.arange(D)
    for b in range(B):
        st, n = min(max(int(start[b]), 0), cap), min(max(int(new[b]), 0), T)
        for first in range(st // 16 * 16, st + n if n else 0, 16):  # (nothing new: nothing is written)
            lo, hi = max(first, st), min(first + 16, st + n)
            pg = int(table[b, first // page]) if first < cap else -1
            here = 0 <= pg < pages
            s0 = first % page
            for h in range(H):
                for i, x in enumerate((k, v)):
                    y = x[b, lo - st:hi - st, h]
                    bad = ~np.isfinite(y).all(-1)
                    e = scale_exponent(np.abs(y[~bad]).max() if (~bad).any() else 0.0)
                    bits = 0
                    if here and lo > first:
                        w = word(want, page, D, pg, h, s0, i)
                        was, bits = old_exponent(w), w & ((1 << (lo - first)) - 1)
                        if was < e:
                            for t in range(lo - first):
                                at = i * page * D + place(D, s0 + t, dims)
                                want[pg, h, at] = code(NUMBERS[want[pg, h, at]] * 2.0 ** (was - e))
                        e = max(e, was)
                    c = code(np.where(bad[:, None], 0.0, y) * 2.0**-e)
                    held[i][b, lo - st:hi - st, h] = np.where(bad[:, None], np.nan, NUMBERS[c] * 2.0**e)
                    for t in range(hi - lo):
                        bits |= int(bad[t]) << (lo - first + t)
                        if here:
                            want[pg, h, i * page * D + place(D, s0 + lo - first + t, dims)] = c[t]
                    if here:
                        at = 2 * page * D + s0 // 16 * 16 + 4 * i
                        want[pg, h, at:at + 4] = np.array([(e + 127) << 23 | bits], np.uint32).view(np.uint8)
    return want, held


def read(cache, table, page, D, b, slots):
    """(codes [n, H, D], scales [n, H, 1]) of keys and of values, float64, NaN scales where a vector is held as NaN; and which tokens are there."""
    dev, H = cache.device, cache.shape[1]
    j = torch.as_tensor(slots, device=dev).long()
    inside = (j >= 0) & (j < table.shape[1] * page)
    j = torch.where(inside, j, 0)
    pg = table[b].long()[j // page]
    there = inside & (pg >= 0) & (pg < cache.shape[0])
    rows = cache[torch.where(there, pg, 0)]  # [n, H, bytes]
    t = (j % page)[:, None, None]
    number = torch.from_numpy(NUMBERS).to(dev)
    out = []
    for i in (0, 1):
        at = i * page * D + place(D, t, torch.arange(D, device=dev))
        c = number[rows.gather(2, at.expand(-1, H, -1)).long()]
        at = 2 * page * D + t // 16 * 16 + 4 * i + torch.arange(4, device=dev)
        w = rows.gather(2, at.expand(-1, H, -1)).contiguous().view(torch.int32).long() & 0xFFFFFFFF
        s = torch.exp2((w >> 23 & 255).double() - 127)
        s = torch.where(w >> (t & 15) & 1 == 1, torch.nan, s)
        out.append((torch.where(there[:, None, None], c, 0.0), torch.where(there[:, None, None], s, 0.0)))
    return out[0], out[1], there


def rotate(x, cos, sin, at, interleaved):
    """x [T, H, D] float64 on the GPU."""
    if cos is None:
        return x
    m = cos.shape[1]
    at = at.clamp(0, cos.shape[0] - 1).long()
    c, s = cos.double()[at][:, None], sin.double()[at][:, None]
    i = torch.arange(m, device=x.device)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + m)
    y = x.clone()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def attention(q, cache, table, start, page, new=None, parent=None, cos=None, sin=None, positions=None, interleaved=False, scale=None):
    """(result, tolerance) [B, T, heads, D] in float64, of GPU tensors.  NaN where the result is."""
    B, T, Hq, D = q.shape
    H = cache.shape[1]
    G, cap, dev = Hq // H, table.shape[1] * page, q.device
    sc = U.sm_scale(D) if scale is None else float(np.float32(scale))
    half, tiny = U.half_step(q.dtype), torch.finfo(q.dtype).smallest_normal * torch.finfo(q.dtype).eps / 2
    lines = torch.from_numpy(U.lines(None if parent is None else parent.cpu().numpy(), T)).to(dev)
    of_q = 0.0 if cos is None and q.dtype == torch.bfloat16 else 2.0**-12
    of_w = 2.0**-8 if q.dtype == torch.bfloat16 else 2.0**-12
    want, tol = torch.zeros((2, B, T, Hq, D), dtype=torch.float64, device=dev)
    for b in range(B):
        before = min(max(int(start[b]), 0), cap)
        fresh = T if new is None else min(max(int(new[b]), 0), T)
        n = min(before + fresh, cap)
        if n == 0:
            continue
        (kc, ks), (vc, vs), there = read(cache, table, page, D, b, range(n))
        bad = (torch.isnan(ks) | torch.isnan(vs))[..., 0]  # [n, H]
        kc, vc, ks, vs = (torch.where(bad[..., None], 0.0, x) for x in (kc, vc, ks, vs))
        at = positions[b] if positions is not None else before + torch.arange(T, device=dev)
        x = rotate(q[b].double(), cos, sin, at, interleaved).reshape(T, H, G, D)
        bad_q = ~torch.isfinite(x).all(-1)
        x = torch.where(bad_q[..., None], 0.0, x)
        see = torch.ones((T, n), dtype=torch.bool, device=dev)
        see[:, before:] = lines[:, :n - before]
        see &= there
        see[fresh:] = False
        nan = (see.double() @ bad.double() > 0)[..., None] | (bad_q & see.any(1)[:, None, None])  # [T, H, G]
        seen = see[None, :, None]  # [1, T, 1, n]
        k, v = kc * ks, vc * vs
        score = torch.einsum("thgd,nhd->htgn", x, k) * sc
        score = torch.where(seen, score, float("-inf"))
        top = score.amax(-1, keepdim=True)
        e = torch.where(seen, torch.exp(score - torch.where(top.isfinite(), top, 0.0)), 0.0)
        total = e.sum(-1, keepdim=True)
        p = torch.where(total > 0, e / total, 0.0)
        mix = lambda w, y: torch.einsum("htgn,nhd->thgd", w, y)  # noqa: E731
        out = mix(p, v)
        # the weights' roundings
        w = p * vs[..., 0].t()[:, None, None]
        pad = (-n) % TILE
        peak = torch.nn.functional.pad(w, (0, pad)).unflatten(-1, (-1, TILE)).amax(-1).repeat_interleave(TILE, -1)[..., :n]
        off = of_w * w + 2.0**-17.5 * peak * (w >= 0)
        err = torch.minimum(mix(off, vc.abs()), 3.5 * mix(off * off, vc * vc).sqrt())
        # the scores' errors, each of which moves its own weight
        far = torch.einsum("thgd,nhd->htgn", x.abs(), k.abs()) * abs(sc)
        row = x.abs().amax(-1)[..., None].permute(1, 0, 2, 3)  # [H, T, G, 1]
        each = of_q * x.abs() + 2.0**-17 * x.abs().amax(-1, keepdim=True) * (x != 0)
        move = torch.minimum(torch.einsum("thgd,nhd->htgn", each, k.abs()), 3.5 * torch.einsum("thgd,nhd->htgn", each * each, k * k).sqrt()) * abs(sc)
        logs = torch.log2(vs.clamp(min=2.0**-40))[..., 0].t()[:, None, None].abs()
        move = move + 2.0**-20 * far + 2.0**-21 * (1 + logs) + 0 * row
        moved = p * torch.expm1(2 * move)
        err = err + mix(moved, v.abs()) + out.abs() * moved.sum(-1).permute(1, 0, 2)[..., None]
        err = err + (TILE + n / TILE) * 2.0**-23 * mix(p, v.abs())
        out, err = (torch.where(nan[..., None], torch.nan, y) for y in (out, (out.abs() + err) * half + err + tiny))
        want[b], tol[b] = out.reshape(T, Hq, D), err.reshape(T, Hq, D)
    return want, tol


def check(got, want, tol):
    """Raises unless got is within tol of want, NaN where want is and nowhere else."""
    x = got.double()
    assert torch.equal(torch.isnan(x), torch.isnan(want)), "NaN in other places"
    over = ((x - want).abs() - tol).nan_to_num(0.0)
    assert bool((over <= 0).all()), f"off by {float((x - want).abs().nan_to_num(0.0).max())}, {float(over.max())} over the tolerance"
