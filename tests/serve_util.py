"""Plain 64-bit forms of the operators around the verification step, for their tests."""
import math

import numpy as np
import torch


# ------------------------------------------------------------------ logit adjustment


def path_of(parent, r):
    """The nodes of row r's context beyond the history: its path without the root."""
    nodes = []
    while r > 0:
        nodes.append(r)
        up = int(parent[r])
        r = up if up < r else 0
    return nodes


def adjust(logits, history=None, lengths=None, prompt_lengths=None, draft_tokens=None, parent=None, repetition=None,
           frequency=None, presence=None, bias_tokens=None, bias_values=None, allowed=None):
    """(result, magnitude of the terms) in float64, from CPU tensors."""
    x = logits.double().numpy()
    B, R, V = x.shape
    out, mag = np.array(x), np.zeros_like(x)
    for b in range(B):
        prompt, output = np.zeros(V, np.int64), np.zeros(V, np.int64)
        if history is not None:
            n = min(max(int(lengths[b]), 0), history.shape[1])
            first = 0 if prompt_lengths is None else int(prompt_lengths[b])
            for i, t in enumerate(history[b, :n].tolist()):
                if 0 <= t < V:
                    (prompt if i < first else output)[t] += 1
        bias = np.zeros(V)
        if bias_tokens is not None:
            for t, v in zip(bias_tokens[b].tolist(), bias_values[b].double().tolist()):
                if 0 <= t < V:
                    bias[t] = v
        rep = 1.0 if repetition is None else float(repetition[b])
        f = 0.0 if frequency is None else float(frequency[b])
        p = 0.0 if presence is None else float(presence[b])
        for r in range(R):
            count = output.copy()
            if draft_tokens is not None:
                for j in (range(r) if parent is None else path_of(parent, r)):
                    t = int(draft_tokens[b, j])
                    if 0 <= t < V:
                        count[t] += 1
            seen = (prompt + count) > 0
            l = np.where(seen, np.where(x[b, r] > 0, x[b, r] / rep, x[b, r] * rep), x[b, r])
            mag[b, r] = np.abs(l) + f * count + abs(p) + np.abs(bias)
            l = l - f * count - p * (count > 0) + bias
            if allowed is not None:
                t = np.arange(V)
                ok = (allowed[b, r].numpy().view(np.uint32)[t // 32] >> (t % 32).astype(np.uint32)) & 1
                l = np.where(ok == 1, l, -np.inf)
            out[b, r] = l
    return out, mag


# ------------------------------------------------------------------------ the cache


def rotate(x, cos, sin, positions, interleaved):
    """x [B, T, H, D] float64; positions [B, T], clamped to the table."""
    if cos is None:
        return x
    m = cos.shape[1]
    at = np.clip(positions, 0, cos.shape[0] - 1)
    c, s = cos[at].astype(np.float64)[:, :, None], sin[at].astype(np.float64)[:, :, None]
    i = np.arange(m)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + m)
    y = np.array(x)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def quantise(x):
    """(codes, scale, zero) of head vectors [..., D] float64; NaN scale and zero for bad ones."""
    with np.errstate(all="ignore"):
        bad = ~np.isfinite(x).all(-1, keepdims=True)
        y = np.where(bad, 0.0, x)
        low, high = y.min(-1, keepdims=True), y.max(-1, keepdims=True)
        zero = np.clip(low, -65504, 65504).astype(np.float32).astype(np.float16) + np.float16(0)  # (-0 is held as +0)
        scale = np.maximum(np.minimum((high - low) / 15, 65504).astype(np.float32).astype(np.float16), np.float16(2.0**-24))
        code = np.clip(np.rint((y - zero.astype(np.float64)) / scale.astype(np.float64)), 0, 15).astype(np.uint8)
    nan = np.float16("nan")
    return np.where(bad, 0, code).astype(np.uint8), np.where(bad, nan, scale), np.where(bad, nan, zero)


def place(page, D, values, token, dim):
    """Half-byte of a code in a page and head, from the documented layout."""
    if not values:
        return token * D + dim
    block, t = divmod(token, 16)
    inside = (((((dim // 32) * 8 + dim % 32 // 4) * 4 + t % 8 // 2) * 2 + t // 8) * 2 + t % 2) * 4 + dim % 4
    return page * D + block * 16 * D + inside


def read_cache(cache, table, page, D, b, n, num_pages):
    """Keys, values [n, H, D] float64 and whether each token is held (page in range), of sequence b."""
    H = cache.shape[1]
    k, v, held = np.zeros((n, H, D)), np.zeros((n, H, D)), np.zeros(n, bool)
    dims = np.arange(D)
    for j in range(n):
        pg, slot = int(table[b, j // page]), j % page
        if not 0 <= pg < num_pages:
            continue
        held[j] = True
        row = cache[pg]
        meta = row[:, page * D:].copy().view(np.float16).reshape(H, 2, page, 2)[:, :, slot].astype(np.float64)
        for i, dst in ((0, k), (1, v)):
            at = np.array([place(page, D, bool(i), slot, int(d)) for d in dims])
            code = (row[:, at // 2] >> (4 * (at % 2)).astype(np.uint8)) & 15
            dst[j] = meta[:, i, 1:] + meta[:, i, :1] * code
    return k, v, held


def attention(q, k, v, see, scale):
    """q [T, Hq, D], k and v [n, H, D], see [T, n]; float64.  Rows that see nothing are 0."""
    T, Hq, D = q.shape
    G = Hq // k.shape[1]
    out = np.zeros((T, Hq, D))
    for t in range(T):
        j = np.nonzero(see[t])[0]
        if not len(j):
            continue
        for h in range(Hq):
            x = scale * (k[j, h // G] @ q[t, h])
            p = np.exp(x - x.max())
            out[t, h] = (p / p.sum()) @ v[j, h // G]
    return out


def lines(parent, T):
    """[T, T]: which new tokens each one sees."""
    m = np.zeros((T, T), bool)
    for i in range(T):
        if parent is None:
            m[i, :i + 1] = True
        else:
            v = i
            while v >= 0:
                m[i, v] = True
                up = int(parent[v])
                v = up if up < v else -1
    return m


def tables(n, pairs, dev="cpu"):
    a = torch.arange(n, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(pairs, dtype=torch.float64) / max(pairs, 1))
    return a.cos().float().to(dev), a.sin().float().to(dev)


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def sm_scale(D):
    return 1 / math.sqrt(D)
