"""The attention over the 4-bit cache in 64 bits on the GPU, with what bounds the kernel's error, element by element.

The kernel's output is sum_j w_j (c_j - 8) + sum_j w_j (z_j + 8 s_j) / s_j over sum_j w_j / s_j, where w_j is p_j s_j times a power of
two of the row's.  Its roundings:
- w_j to fp16 before the first sum, by 2^-11 of itself, and once more where the row's power of two moves: at most
  2 * 2^-11 sum_j p_j s_j |c_j - 8|.  They are independent, each uniform within its half step (a deviation of 2^-11 / sqrt(3)), so
  that six deviations of the sum of both are 4.9 * 2^-11 sqrt(sum_j (p_j s_j (c_j - 8))^2);
- weights below fp16's normal range, by 2^-25 where the largest is at least 2^7: 2^-32 of it, 8 times that in the output, twice;
- scores: fp32 sums of D products of fp16 numbers, taken 16 at a time (D / 16 steps of 2^-23 of their size) and a few roundings
  more (the exponential's, logarithm's and reciprocal's 2^-22 among them): (D / 16 + 4) 2^-23 of scale sum_d |q_d| (s |c_d - 8| +
  |z + 8 s|), which bounds the score itself; each moves its own weight;
- a rotated bf16 query to 11 bits: 2^-11 scale sum_d |q_d k_d|;
- the sums in fp32: of the weights' products 8 steps a unit, `units` of them in a row, and of the joins at most 16: 2^-23 each of their
  terms' sizes;
- the output to its type."""
import torch

from tests import serve_util as U


def read(cache, table, page, D, b, n):
    """codes [n, H, D], scales and zeros [n, H, 1] of keys and values (float64), and which tokens are held, of sequence b."""
    dev, H = cache.device, cache.shape[1]
    j = torch.arange(n, device=dev)
    pg = table[b].long()[j // page]
    held = (pg >= 0) & (pg < cache.shape[0])
    rows = cache[torch.where(held, pg, 0)]  # [n, H, bytes]
    t = j % page
    out = []
    for i in (0, 1):
        at = torch.tensor([[U.place(page, D, bool(i), s, d) for d in range(D)] for s in range(page)], device=dev)[t][:, None].expand(n, H, D)
        code = (rows.gather(2, at // 2) >> (4 * (at % 2)).to(torch.uint8)) & 15
        o = (page * D + i * 4 * page + 4 * t)[:, None, None] + torch.arange(4, device=dev)
        sz = rows.gather(2, o.expand(n, H, 4)).contiguous().view(torch.float16).double()
        out.append(tuple(torch.where(held[:, None, None], y, 0.0) for y in (code.double(), sz[..., :1], sz[..., 1:])))
    return out[0], out[1], held


def rotate(x, cos, sin, at, interleaved):
    """x [T, H, D] float64."""
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


def attention(q, cache, table, start, page, new=None, parent=None, cos=None, sin=None, positions=None, interleaved=False, scale=None, units=8):
    """(result, tolerance) [B, T, heads, D] in float64, of GPU tensors."""
    B, T, Hq, D = q.shape
    H = cache.shape[1]
    G, cap, dev = Hq // H, table.shape[1] * page, q.device
    sc = U.sm_scale(D) if scale is None else scale
    half, tiny = U.half_step(q.dtype), torch.finfo(q.dtype).smallest_normal * torch.finfo(q.dtype).eps / 2
    lines = torch.from_numpy(U.lines(None if parent is None else parent.cpu().numpy(), T)).to(dev)
    want, tol = torch.zeros((2, B, T, Hq, D), dtype=torch.float64, device=dev)
    for b in range(B):
        before = min(max(int(start[b]), 0), cap)
        fresh = T if new is None else min(max(int(new[b]), 0), T)
        n = min(before + fresh, cap)
        if n == 0:
            continue
        (kc, ks, kz), (vc, vs, vz), held = read(cache, table, page, D, b, n)
        at = positions[b] if positions is not None else before + torch.arange(T, device=dev)
        x = rotate(q[b].double(), cos, sin, at, interleaved).reshape(T, H, G, D)
        see = torch.ones((T, n), dtype=torch.bool, device=dev)
        see[:, before:] = lines[:, :n - before]
        see &= held
        see[fresh:] = False
        see = see[None, :, None]  # [1, T, 1, n]
        k, v = kz + ks * kc, vz + vs * vc
        score = torch.einsum("thgd,nhd->htgn", x, k) * sc
        score = torch.where(see, score, float("-inf"))
        top = score.amax(-1, keepdim=True)
        e = torch.where(see, torch.exp(score - torch.where(top.isfinite(), top, 0.0)), 0.0)
        total = e.sum(-1, keepdim=True)
        p = torch.where(total > 0, e / total, 0.0)
        mix = lambda w, y: torch.einsum("htgn,nhd->thgd", w, y)  # noqa: E731
        out = mix(p, v)
        code = vs * (vc - 8)
        linear, square = mix(p, code.abs()), mix(p * p, code * code).sqrt()
        peak = (p * vs[..., 0].t()[:, None, None]).amax(-1).permute(1, 0, 2)[..., None]  # [T, H, G, 1]
        far = torch.einsum("thgd,nhd->htgn", x.abs(), (ks * (kc - 8)).abs() + (kz + 8 * ks).abs()) * abs(sc)
        move = (D / 16 + 4) * 2.0**-23 * far + 2.0**-21
        if cos is not None and q.dtype == torch.bfloat16:
            move = move + 2.0**-11 * torch.einsum("thgd,nhd->htgn", x.abs(), k.abs()) * abs(sc)
        moved = p * torch.expm1(2 * move)
        err = torch.minimum(2 * 2.0**-11 * linear, 4.9 * 2.0**-11 * square) + n * 2.0**-28 * peak
        err = err + mix(moved, v.abs()) + out.abs() * moved.sum(-1).permute(1, 0, 2)[..., None]
        err = err + (8 * units + 16) * 2.0**-23 * (linear + mix(p, (vz + 8 * vs).abs().expand_as(v)))
        want[b], tol[b] = out.reshape(T, Hq, D), (err + (out.abs() + err) * half + tiny).reshape(T, Hq, D)
    return want, tol
