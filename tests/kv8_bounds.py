"""spec_kv8_attention in 64 bits with a tolerance that holds token by token: no token's error is measured by another one's size.

With p_j the probabilities and v_j the held values, the result of dimension d is sum_j p_j v_jd, and what it may be off by is
- a weight, p_j times its value's scale, is held in parts that have 11 bits for bf16 outputs and 15 for fp16 ones, at the lower end of a range of
  exponents 2^-8.5 and 2^-11.9 of itself; its last part's smallest step is less than 2^-51.5 of the largest weight among the 128 tokens of its tile;
- a score's error moves its own weight, by as much relatively.  The queries' parts (kv8_reference.py derives these numbers): 2^-12 of a number
  unless it is bf16 and not rotated, and 2^-17 of its row's largest one; the fp32 sums of products: 2^-20 of the sum of their sizes; the shift by
  log2 s' and the maximum, and the exponential: 2^-21 (1 + |log2 s'|).  Within six deviations as there.  A moved weight moves the sum of weights too;
- sums in fp32: 2^-23 each of the sum of sizes, 128 + tiles of them at most, in the weights' sum as well;
- the output is rounded to its type.
All but the smallest step are shares of sum_j p_j |v_jd|, and of the result, which is not larger.  Tokens that a row does not see add nothing."""
import torch

from tests import kv8_reference as R
from tests import serve_util as U


def attention(q, cache, table, start, page, new=None, parent=None, cos=None, sin=None, positions=None, scale=None):
    """(result, tolerance, sum p |v|) [B, T, heads, D] in float64, of GPU tensors without NaN."""
    B, T, Hq, D = q.shape
    H = cache.shape[1]
    G, cap, dev = Hq // H, table.shape[1] * page, q.device
    sc = U.sm_scale(D) if scale is None else scale
    half, tiny = U.half_step(q.dtype), torch.finfo(q.dtype).smallest_normal * torch.finfo(q.dtype).eps / 2
    lines = torch.from_numpy(U.lines(None if parent is None else parent.cpu().numpy(), T)).to(dev)
    of_w = 2.0**-8.5 if q.dtype == torch.bfloat16 else 2.0**-11.9
    of_q = 0.0 if cos is None and q.dtype == torch.bfloat16 else 2.0**-12
    want, tol, size = torch.zeros((3, B, T, Hq, D), dtype=torch.float64, device=dev)
    for b in range(B):
        before = int(start[b])
        fresh = T if new is None else int(new[b])
        n = min(before + fresh, cap)
        if n == 0 or fresh == 0:
            continue
        (kc, ks), (vc, vs), there = R.read(cache, table, page, D, b, range(n))
        k, v = kc * ks, vc * vs
        at = positions[b] if positions is not None else before + torch.arange(T, device=dev)
        x = R.rotate(q[b].double(), cos, sin, at, False).reshape(T, H, G, D)
        see = torch.ones((T, n), dtype=torch.bool, device=dev)
        see[:, before:] = lines[:, :n - before]
        see &= there
        see[fresh:] = False
        seen = see[None, :, None]
        score = torch.where(seen, torch.einsum("thgd,nhd->htgn", x, k) * sc, float("-inf"))
        e = torch.exp(score - score.amax(-1, keepdim=True).nan_to_num(0.0, 0.0, 0.0))
        total = e.sum(-1, keepdim=True)
        p = torch.where(total > 0, e / total, 0.0)
        mix = lambda w, y: torch.einsum("htgn,nhd->thgd", w, y)  # noqa: E731
        out, most = mix(p, v), mix(p, v.abs())
        each = of_q * x.abs() + 2.0**-17 * x.abs().amax(-1, keepdim=True) * (x != 0)
        move = torch.minimum(torch.einsum("thgd,nhd->htgn", each, k.abs()), 3.5 * torch.einsum("thgd,nhd->htgn", each**2, k**2).sqrt()) * abs(sc)
        move = move + 2.0**-20 * torch.einsum("thgd,nhd->htgn", x.abs(), k.abs()) * abs(sc)
        move = move + 2.0**-21 * (1 + torch.log2(vs.clamp(min=2.0**-40))[..., 0].t()[:, None, None].abs())
        moved = p * torch.expm1(2 * move)
        w = p * vs[..., 0].t()[:, None, None]
        peak = torch.nn.functional.pad(w, (0, -n % R.TILE)).unflatten(-1, (-1, R.TILE)).amax(-1).repeat_interleave(R.TILE, -1)[..., :n]
        step = 2.0**-51.5 * mix(torch.where(seen, peak, 0.0), vc.abs())
        sums = (R.TILE + n / R.TILE) * 2.0**-23
        err = mix(moved, v.abs()) + out.abs() * moved.sum(-1).permute(1, 0, 2)[..., None] + (of_w + 2 * sums) * most + step
        want[b], tol[b], size[b] = (y.reshape(T, Hq, D) for y in (out, (out.abs() + err) * half + err + tiny, most))
    return want, tol, size
