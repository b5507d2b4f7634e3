"""The operators around the verification step: what they compute, on real sizes.

Three operators, each in a plain form (elementary torch operations) and as the call that a
user of the package makes:

  adjust   penalties for repeated tokens, biases and grammar masks on the logits of the
           verified rows (chain or token tree)
  append   the new tokens' keys and values into a paged cache held in 4 bits, the position
           rotation applied on the way; gives back the values that the cache holds for them
  attend   the new tokens' attention (chain or tree) over that cache

The cache is [pages][heads][page_size * (D + 8)] bytes.  Per page and head: the keys'
codes, the values' codes, then (scale, zero) as two fp16 per token for the keys and for the
values.  A key's codes lie in the order of its dimensions, two to a byte, the lower first.  The
values' codes lie in blocks of 16 tokens, [D/32][8 (d%32)/4][4 (tok%8)/2][2 tok/8][2 tok%2][2 bytes
of 2 codes].  With x the head's (rotated) vector: zero = fp16(min x), scale = fp16((max x - min x) / 15),
at least 2^-24, code = round((x - zero) / scale) clamped to 0..15, and the value held is zero + scale * code.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------------------- cases


def listed():
    return [
        # the smallest verification call: one sequence, four drafts, a toy vocabulary
        dict(name="adjust_b1", op="adjust", B=1, rows=5, V=1000, dtype="fp32", tree=False, history=200, bias=0, grammar=False),
        # a serving batch of chat requests with penalties and a few biased tokens each
        dict(name="adjust_b64", op="adjust", B=64, rows=6, V=32000, dtype="bf16", tree=False, history=2000, bias=32, grammar=False),
        # a full batch on a large vocabulary, part of it held to a grammar
        dict(name="adjust_b256", op="adjust", B=256, rows=9, V=128256, dtype="bf16", tree=False, history=1500, bias=16, grammar=True),
        # every node of a token tree, an odd vocabulary (rows off the 16-byte grid), long histories
        dict(name="adjust_tree", op="adjust", B=64, rows=64, V=50257, dtype="fp32", tree=True, history=4001, bias=8, grammar=True),
        # one sequence decoding one token
        dict(name="append_b1", op="append", B=1, T=1, Hkv=8, D=128, dtype="bf16", page=16, L=700, rotary=128, interleaved=False, ragged=False),
        # eight drafts and the last token of a full batch
        dict(name="append_b256", op="append", B=256, T=9, Hkv=8, D=128, dtype="bf16", page=64, L=4096, rotary=128, interleaved=False, ragged=False),
        # prompts of odd lengths taken in at once, a rotation over part of the head in neighbouring pairs
        dict(name="append_prompt", op="append", B=8, T=2001, Hkv=16, D=64, dtype="fp16", page=32, L=100, rotary=32, interleaved=True, ragged=True),
        # one sequence decoding one token
        dict(name="attend_b1", op="attend", B=1, T=1, Hq=32, Hkv=8, D=128, dtype="bf16", page=16, L=700, tree=False, rope=True, ragged=False),
        # verifying eight drafts of a batch with contexts of all lengths
        dict(name="attend_chain", op="attend", B=64, T=9, Hq=32, Hkv=8, D=128, dtype="bf16", page=64, L=4096, tree=False, rope=True, ragged=True),
        # verifying a token tree of 64 nodes
        dict(name="attend_tree", op="attend", B=64, T=64, Hq=16, Hkv=4, D=64, dtype="fp16", page=32, L=2047, tree=True, rope=False, ragged=True),
        # a large batch decoding single tokens over long contexts
        dict(name="attend_b256", op="attend", B=256, T=1, Hq=64, Hkv=8, D=128, dtype="bf16", page=64, L=8192, tree=False, rope=True, ragged=True),
        # five drafts over one very long context, wide heads
        dict(name="attend_long", op="attend", B=1, T=6, Hq=16, Hkv=4, D=256, dtype="bf16", page=128, L=200001, tree=False, rope=True, ragged=False),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["adjust", "append", "attend"])
    if op == "adjust":
        tree = rng.random() < 0.3
        V, B = _logint(rng, 1000, 152064), _logint(rng, 1, 256)
        rows = rng.randint(2, 64) if tree else rng.randint(1, 12)
        while B * rows * V > 280_000_000:
            B = max(1, B // 2)
            rows = rows if B > 1 else max(1, rows // 2)
        return dict(op=op, B=B, rows=rows, V=V, dtype=rng.choice(["bf16", "fp32"]), tree=tree, history=_logint(rng, 1, 8000),
                    bias=rng.choice([0, 1, 17, 64, 300]), grammar=rng.random() < 0.5)
    D = rng.choice([64, 128, 256])
    Hkv = rng.choice([1, 2, 4, 5, 8, 16])
    page, dtype = rng.choice([16, 32, 48, 64, 128]), rng.choice(["bf16", "fp16"])
    if op == "append":
        B, T = _logint(rng, 1, 256), _logint(rng, 1, 2500)
        while B * T * Hkv * D > 16_000_000:
            T = max(1, T // 2)
            B = B if T > 1 else max(1, B // 2)
        return dict(op=op, B=B, T=T, Hkv=Hkv, D=D, dtype=dtype, page=page, L=_logint(rng, 1, 8000), rotary=rng.choice([D, D, D // 2, 0]),
                    interleaved=rng.random() < 0.4, ragged=rng.random() < 0.5)
    tree = rng.random() < 0.3
    G = rng.choice([1, 2, 3, 4, 7, 8])
    B, T, L = _logint(rng, 1, 256), rng.randint(2, 64) if tree else rng.choice([1, 1, 2, 4, 6, 9, 17]), _logint(rng, 16, 100000)
    while B * L * Hkv * D > 1_000_000_000 or B * L * Hkv * G * T > 300_000_000:
        B, L = (B // 2, L) if B > 8 or (B > 1 and L < 64) else (B, L // 2)
    return dict(op=op, B=max(1, B), T=T, Hq=Hkv * G, Hkv=Hkv, D=D, dtype=dtype, page=page, L=max(1, L), tree=tree, rope=rng.random() < 0.5, ragged=rng.random() < 0.6)


# ------------------------------------------------------------------------------ inputs


def _parents(n, gen):
    """A token tree: parents before children, mostly a few levels deep; node 0 is the root."""
    at = torch.arange(1, n)
    back = torch.minimum((torch.rand(n - 1, generator=gen) ** 0.7 * (n / 2 + 1)).long() + 1, at)
    return torch.cat([torch.tensor([-1]), at - back]).to(torch.int32)


def _tables(positions, rotary):
    angle = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * (
        10000.0 ** (-torch.arange(rotary // 2, dtype=torch.float64, device="cuda") * 2 / max(rotary, 1)))
    return angle.cos().float(), angle.sin().float()


def _heads(n, H, D, gen, offsets):
    """Head vectors with the few strong channels that keys have (offsets [H, D])."""
    return torch.randn((n, H, D), device="cuda", generator=gen) + offsets


def prepare(case, seed):
    c, dev = case, "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    s = dict(case=c)
    if c["op"] == "adjust":
        B, R, V, n = c["B"], c["rows"], c["V"], c["history"]
        s["logits"] = (torch.randn((B, R, V), device=dev, generator=gen) * 3).to(DT[c["dtype"]])
        # tokens as text has them: a few very often
        words = lambda *shape: ((torch.rand(shape, device=dev, generator=gen) ** 4) * V).clamp(max=V - 1).to(torch.int32)  # noqa: E731
        s["history"], s["draft_tokens"] = words(B, n), words(B, R if c["tree"] else R - 1)
        s["lengths"] = torch.randint(n // 2, n + 1, (B,), generator=host).to(dev, torch.int32)
        s["prompt_lengths"] = (s["lengths"] * torch.rand(B, device=dev, generator=gen)).to(torch.int32)
        s["parent"] = _parents(R, host).to(dev) if c["tree"] else None
        s["repetition"] = 1 + 0.3 * torch.rand(B, device=dev, generator=gen)
        s["frequency"] = 0.5 * torch.rand(B, device=dev, generator=gen)
        s["presence"] = torch.rand(B, device=dev, generator=gen)
        k = c["bias"]
        s["bias_tokens"] = torch.randint(0, V, (B, k), generator=host).to(dev, torch.int32) if k else None
        s["bias_values"] = 4 * torch.randn((B, k), device=dev, generator=gen) if k else None
        s["allowed"] = None
        if c["grammar"]:  # a third of the rows free, a third with a broad class of tokens, a third with few
            w = (V + 31) // 32
            bits = lambda: torch.randint(-2**31, 2**31 - 1, (B, R, w), device=dev, generator=gen, dtype=torch.int64).to(torch.int32)  # noqa: E731
            kind = torch.randint(0, 3, (B, R, 1), device=dev, generator=gen)
            few = bits() & bits() & bits() & bits() & bits()
            s["allowed"] = torch.where(kind == 0, torch.full_like(few, -1), torch.where(kind == 1, bits(), few))
        return s
    B, T, Hkv, D, page, L = c["B"], c["T"], c["Hkv"], c["D"], c["page"], c["L"]
    dt = DT[c["dtype"]]
    start = torch.randint(L // 8, L + 1, (B,), generator=host) if c["ragged"] else torch.full((B,), L)
    s["new_lens"] = torch.randint((T + 1) // 2, T + 1, (B,), generator=host).to(dev, torch.int32) if c["op"] == "append" and c["ragged"] else None
    width = (L + T + page - 1) // page
    pages = B * width + 3
    s["page_table"] = torch.randperm(pages, generator=host)[:B * width].reshape(B, width).to(dev, torch.int32)
    s["start"] = start.to(dev, torch.int32)
    s["cache"] = torch.zeros((pages, Hkv, page * (D + 8)), dtype=torch.uint8, device=dev)
    rotary = c["rotary"] if c["op"] == "append" else D if c["rope"] else 0
    s["cos"], s["sin"] = _tables(L + T, rotary) if rotary else (None, None)
    s["positions"], s["parent"] = None, None
    offsets = 4 * torch.randn((Hkv, D), device=dev, generator=gen) * (torch.rand((Hkv, D), device=dev, generator=gen) < 0.04)
    if c["op"] == "append":
        s["k"] = _heads(B * T, Hkv, D, gen, offsets).reshape(B, T, Hkv, D).to(dt)
        s["v"] = _heads(B * T, Hkv, D, gen, 0.0).reshape(B, T, Hkv, D).to(dt)
        return s
    if c["tree"]:
        s["parent"] = _parents(T, host).to(dev)
        depth = _ancestors(s["parent"]).sum(1) - 1
        s["positions"] = (s["start"][:, None] + depth[None, :]).to(torch.int32)
    s["q"] = torch.randn((B, T, c["Hq"], D), device=dev, generator=gen).to(dt)
    # the whole pool is filled, a part at a time: pages that no sequence reads hold old tokens
    step = max(1, 400_000_000 // (Hkv * page * D * 8))
    for p in range(0, pages, step):
        n = min(step, pages - p)
        k = _heads(n * page, Hkv, D, gen, offsets).transpose(0, 1)
        v = _heads(n * page, Hkv, D, gen, 0.0).transpose(0, 1)
        (kc, ks, kz), (vc, vs, vz) = _quantise(k), _quantise(v)
        s["cache"][p:p + n] = _pack(*(x.reshape(Hkv, n, page, -1).transpose(0, 1) for x in (kc, ks, kz, vc, vs, vz)))
    return s


# ------------------------------------------------------------------------- plain forms


def _ancestors(parent):
    """[N, N] truth values: whether node j is on the path from the root to node i (itself too)."""
    n = parent.numel()
    reach = torch.eye(n, device=parent.device)
    up = torch.zeros((n, n), device=parent.device)
    up[torch.arange(1, n), parent[1:].long()] = 1
    for _ in range(max(1, n.bit_length())):  # paths of length 1, 2, 4, ..
        reach = ((reach + up @ reach) > 0).float()
        up = ((up @ up) > 0).float()
    return reach > 0


def _quantise(x):
    """Codes (uint8) of x [..., D] and its (scale, zero), held in fp16; in x's own precision."""
    low, high = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    zero = low.to(torch.float16)
    scale = ((high - low) / 15).to(torch.float16).clamp(min=2.0**-24)
    code = ((x - zero.to(x.dtype)) / scale.to(x.dtype)).round().clamp(0, 15)
    return code.to(torch.uint8), scale, zero


def _pack(kc, ks, kz, vc, vs, vz):
    """Page bytes [n, H, page * (D + 8)] of codes [n, H, page, D] and scales [n, H, page, 1]."""
    n, H, page, D = kc.shape
    kb = (kc[..., 0::2] | (kc[..., 1::2] << 4)).reshape(n, H, -1)
    vb = vc[..., 0::2] | (vc[..., 1::2] << 4)  # [n, H, page, D / 2]
    vb = vb.reshape(n, H, page // 16, 2, 4, 2, D // 32, 8, 2).permute(0, 1, 2, 6, 7, 4, 3, 5, 8).reshape(n, H, -1)
    meta = lambda a, b: torch.cat([a, b], -1).contiguous().view(torch.uint8).reshape(n, H, -1)  # noqa: E731
    return torch.cat([kb, vb, meta(ks, kz), meta(vs, vz)], -1)


def _unpack(b, page, D, dt):
    """Keys and values [n, H, page, D] that page bytes [n, H, page * (D + 8)] stand for."""
    n, H, half = b.shape[0], b.shape[1], page * D // 2
    two = lambda x: torch.stack([x & 15, x >> 4], -1)  # noqa: E731
    kc = two(b[..., :half]).reshape(n, H, page, D)
    vc = two(b[..., half:2 * half]).reshape(n, H, page // 16, D // 32, 8, 4, 2, 2, 2, 2)
    vc = vc.permute(0, 1, 2, 6, 5, 7, 3, 4, 8, 9).reshape(n, H, page, D)
    meta = b[..., 2 * half:].contiguous().view(torch.float16).reshape(n, H, 2, page, 2, 1).to(dt)
    return kc.to(dt) * meta[:, :, 0, :, 0] + meta[:, :, 0, :, 1], vc.to(dt) * meta[:, :, 1, :, 0] + meta[:, :, 1, :, 1]


def _rotate(x, cos, sin, at, interleaved):
    """x [B, T, H, D] with its first 2 * cos.shape[1] dimensions turned by the angles of positions at [B, T]."""
    if cos is None:
        return x
    m = cos.shape[1]
    c, s = cos[at.long()][:, :, None].to(x.dtype), sin[at.long()][:, :, None].to(x.dtype)
    a, b = (x[..., 0:2 * m:2], x[..., 1:2 * m:2]) if interleaved else (x[..., :m], x[..., m:2 * m])
    a, b = a * c - b * s, b * c + a * s
    turned = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([turned, x[..., 2 * m:]], -1)


def _adjust(s):
    c = s["case"]
    B, R, V, n = c["B"], c["rows"], c["V"], c["history"]
    dev = s["logits"].device
    at = torch.arange(n, device=dev)[None]
    inside, said = at < s["lengths"][:, None], (at < s["lengths"][:, None]) & (at >= s["prompt_lengths"][:, None])
    h = s["history"].long()
    seen = torch.zeros((B, V), dtype=torch.int32, device=dev).scatter_add_(1, h, inside.int())
    count = torch.zeros((B, V), dtype=torch.int32, device=dev).scatter_add_(1, h, said.int())
    if c["tree"]:
        on = _ancestors(s["parent"]).int()
        on[:, 0] = 0  # the root is the last token of the history
    else:
        on = torch.ones((R, R - 1), dtype=torch.int32, device=dev).tril(-1)
    J = on.shape[1]
    more = torch.zeros((B, R, V), dtype=torch.int32, device=dev).scatter_add_(
        2, s["draft_tokens"].long()[:, None].expand(B, R, J), on[None].expand(B, R, J))
    count = count[:, None] + more
    seen = seen[:, None] + more
    x = s["logits"].float()
    each = lambda name: s[name][:, None, None]  # noqa: E731
    x = torch.where(seen > 0, torch.where(x > 0, x / each("repetition"), x * each("repetition")), x)
    x = x - each("frequency") * count - each("presence") * (count > 0)
    if s["bias_tokens"] is not None:
        k = c["bias"]
        rank = torch.zeros((B, V), dtype=torch.int64, device=dev).scatter_reduce_(
            1, s["bias_tokens"].long(), torch.arange(1, k + 1, device=dev)[None].expand(B, k), "amax")
        bias = torch.cat([torch.zeros((B, 1), device=dev), s["bias_values"]], 1).gather(1, rank)  # the last entry of a token counts
        x = x + bias[:, None]
    if s["allowed"] is not None:
        bit = (s["allowed"][..., None] >> torch.arange(32, device=dev, dtype=torch.int32)) & 1
        x = torch.where(bit.flatten(-2)[..., :V] == 1, x, float("-inf"))
    return x.to(s["logits"].dtype)


def _append(s):
    c = s["case"]
    B, T, Hkv, D, page = c["B"], c["T"], c["Hkv"], c["D"], c["page"]
    dev, dt = s["k"].device, s["k"].dtype
    slot = s["start"][:, None].long() + torch.arange(T, device=dev)
    live = torch.ones((B, T), dtype=torch.bool, device=dev) if s["new_lens"] is None else torch.arange(T, device=dev) < s["new_lens"][:, None]
    # codes near a border between two need more than 32 bits
    kc, ks, kz = _quantise(_rotate(s["k"].double(), s["cos"], s["sin"], slot, c["interleaved"]))
    vc, vs, vz = _quantise(s["v"].double())
    b, t = live.nonzero(as_tuple=True)
    where = slot[b, t]
    pg, tok = s["page_table"].long()[b, where // page], where % page
    d, head = torch.arange(D // 2, device=dev), torch.arange(Hkv, device=dev)[None, :, None]
    pg, tok = pg[:, None, None], tok[:, None, None]
    two = lambda x: x[b, t][..., 0::2] | (x[b, t][..., 1::2] << 4)  # noqa: E731
    half, e = page * D // 2, 2 * d
    in_block = (e // 32) * 256 + ((e % 32) // 4 * 4 + tok % 8 // 2) * 8 + tok % 16 // 8 * 4 + tok % 2 * 2 + e % 4 // 2
    s["cache"][pg, head, tok * (D // 2) + d] = two(kc)
    s["cache"][pg, head, half + tok // 16 * (8 * D) + in_block] = two(vc)
    four = torch.arange(4, device=dev)
    s["cache"][pg, head, 2 * half + tok * 4 + four] = torch.cat([ks, kz], -1)[b, t].contiguous().view(torch.uint8)
    s["cache"][pg, head, 2 * half + 4 * page + tok * 4 + four] = torch.cat([vs, vz], -1)[b, t].contiguous().view(torch.uint8)
    held = lambda code, scale, zero: torch.where(live[..., None, None], zero.float() + scale.float() * code.float(), 0.0).to(dt)  # noqa: E731
    return held(kc, ks, kz), held(vc, vs, vz)


def _attend(s):
    c = s["case"]
    B, T, Hq, Hkv, D, page = c["B"], c["T"], c["Hq"], c["Hkv"], c["D"], c["page"]
    dev, dt = s["q"].device, s["q"].dtype
    at = s["positions"] if s["positions"] is not None else s["start"][:, None] + torch.arange(T, device=dev)
    q = _rotate(s["q"].float(), s["cos"], s["sin"], at, False).reshape(B, T, Hkv, Hq // Hkv, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D)
    width = s["page_table"].shape[1]
    k, v = _unpack(s["cache"][s["page_table"].flatten().long()], page, D, torch.float32)
    k, v = (x.reshape(B, width, Hkv, page, D).transpose(1, 2).reshape(B, Hkv, width * page, D) for x in (k, v))
    j = torch.arange(width * page, device=dev) - s["start"][:, None]  # [B, L], below 0: before the new tokens
    among = _ancestors(s["parent"]) if c["tree"] else torch.ones((T, T), dtype=torch.bool, device=dev).tril()
    new = among[:, j.clamp(0, T - 1)].transpose(0, 1)  # [B, T, L]
    see = ((j < 0)[:, None] | (new & ((j >= 0) & (j < T))[:, None]))[:, None, :, None]  # [B, 1, T, 1, L]
    x = (q @ k.transpose(-1, -2) / math.sqrt(D)).reshape(B, Hkv, T, Hq // Hkv, -1)
    x = torch.where(see, x, float("-inf"))
    p = torch.exp(x - x.amax(-1, keepdim=True))
    p = (p / p.sum(-1, keepdim=True)).reshape(B, Hkv, T * (Hq // Hkv), -1)
    return (p @ v).reshape(B, Hkv, T, -1, D).transpose(1, 2).reshape(B, T, Hq, D).to(dt)


# --------------------------------------------------------------------------- the calls


def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return _adjust(s) if op == "adjust" else _append(s) if op == "append" else _attend(s)
    import speculative_decoding_verify_spec_gb300 as sv
    if op == "adjust":
        return sv.spec_logit_adjust(s["logits"], history=s["history"], lengths=s["lengths"], prompt_lengths=s["prompt_lengths"],
                                    draft_tokens=s["draft_tokens"], parent=s["parent"], repetition=s["repetition"],
                                    frequency=s["frequency"], presence=s["presence"], bias_tokens=s["bias_tokens"],
                                    bias_values=s["bias_values"], allowed=s["allowed"])
    if op == "append":
        return sv.spec_kv_append(s["k"], s["v"], s["cache"], s["page_table"], s["start"], new_lens=s["new_lens"], cos=s["cos"],
                                 sin=s["sin"], interleaved=s["case"]["interleaved"], return_values=True)
    return sv.spec_kv_attention(s["q"], s["cache"], s["page_table"], s["start"], parent=s["parent"], cos=s["cos"], sin=s["sin"],
                                positions=s["positions"])


# ---------------------------------------------------------------- in 64 bits, and costs


def _exact_adjust(s):
    c = s["case"]
    B, R, V = c["B"], c["rows"], c["V"]
    out = s["logits"].double()
    lens, firsts = s["lengths"].tolist(), s["prompt_lengths"].tolist()
    up = s["parent"].tolist() if c["tree"] else None
    for b in range(B):
        h = s["history"][b, :lens[b]].long()
        prompt = torch.bincount(h[:firsts[b]], minlength=V)
        output = torch.bincount(h[firsts[b]:], minlength=V)
        for r in range(R):
            path = []
            if up is None:
                path = list(range(r))
            else:
                while r > 0 and (not path or up[path[-1]] > 0):
                    path.append(r if not path else up[path[-1]])
            n = output if not path else output + torch.bincount(s["draft_tokens"][b, path].long(), minlength=V)
            x, rep = out[b, r], s["repetition"][b].double()
            hit = (prompt + n) > 0
            x[hit] = torch.where(x[hit] > 0, x[hit] / rep, x[hit] * rep)
            x -= s["frequency"][b].double() * n + s["presence"][b].double() * (n > 0)
        if s["bias_tokens"] is not None:
            last = dict(zip(s["bias_tokens"][b].tolist(), range(c["bias"])))
            out[b][:, list(last)] += s["bias_values"][b, list(last.values())].double()
    if s["allowed"] is not None:
        token = torch.arange(V, device=out.device)
        for b in range(B):
            out[b][((s["allowed"][b][:, token // 32] >> (token % 32)) & 1) == 0] = -math.inf
    return out


def _exact_append(s):
    c = s["case"]
    k, v = s["k"].double().clone(), s["v"].double()
    T, at = c["T"], s["start"][:, None].long() + torch.arange(c["T"], device="cuda")
    for i in range(0 if s["cos"] is None else s["cos"].shape[1]):
        a, b = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + s["cos"].shape[1])
        turn = torch.complex(s["cos"][at, i].double(), s["sin"][at, i].double())[..., None]
        z = torch.complex(k[..., a], k[..., b]) * turn
        k[..., a], k[..., b] = z.real, z.imag
    held = []
    for x in (k, v):
        zero = x.min(-1, keepdim=True)[0].half().double()
        scale = ((x.max(-1, keepdim=True)[0] - x.min(-1, keepdim=True)[0]) / 15).half().double().clamp(min=2.0**-24)
        y = zero + scale * torch.clamp(torch.round((x - zero) / scale), 0, 15)
        if s["new_lens"] is not None:
            y[torch.arange(T, device="cuda")[None] >= s["new_lens"][:, None]] = 0
        held.append(y)
    return tuple(held)


def _exact_attend(s):
    c = s["case"]
    B, T, Hq, Hkv, D, page = c["B"], c["T"], c["Hq"], c["Hkv"], c["D"], c["page"]
    G, half = Hq // Hkv, page * D // 2
    start, up = s["start"].tolist(), s["parent"].tolist() if c["tree"] else [i - 1 for i in range(T)]
    lines = torch.zeros((T, T), dtype=torch.bool, device="cuda")
    for i in range(T):
        if i:
            lines[i] = lines[up[i]]
        lines[i, i] = True
    out = torch.empty((B, T, Hq, D), dtype=torch.float64, device="cuda")
    d = torch.arange(D, device="cuda")
    for b in range(B):
        n = start[b] + T
        tok = torch.arange(n, device="cuda")
        rows = s["cache"][s["page_table"][b, :(n + page - 1) // page].long()].transpose(0, 1)  # [H, pages, bytes]
        scales = rows[..., 2 * half:].contiguous().view(torch.float16).double().reshape(Hkv, -1, 2, page, 2)
        rows = rows.reshape(Hkv, -1)
        base, t = tok // page * (page * (D + 8)), tok % page
        kbyte = (base + t * (D // 2))[:, None] + d // 2
        vbyte = (base + half + t // 16 * (8 * D) + t % 8 // 2 * 8 + t % 16 // 8 * 4 + t % 2 * 2)[:, None] + d // 32 * 256 + d % 32 // 4 * 32 + d % 4 // 2
        held = []
        for i, byte in enumerate((kbyte, vbyte)):
            code = (rows[:, byte] >> (4 * (d % 2)).to(torch.uint8)) & 15
            sz = scales[:, :, i].reshape(Hkv, -1, 2)[:, :n]
            held.append(sz[..., 1:] + sz[..., :1] * code)
        q = s["q"][b].double()
        if s["cos"] is not None:
            at = (s["positions"][b] if s["positions"] is not None else start[b] + torch.arange(T, device="cuda")).long()
            z = torch.complex(q[..., :D // 2], q[..., D // 2:]) * torch.complex(s["cos"][at].double(), s["sin"][at].double())[:, None]
            q = torch.cat([z.real, z.imag], -1)
        x = torch.einsum("thgd,hnd->htgn", q.reshape(T, Hkv, G, D), held[0]) / math.sqrt(D)
        x[..., start[b]:].masked_fill_(~lines[None, :, None], -math.inf)
        out[b] = torch.einsum("htgn,hnd->thgd", torch.softmax(x, -1), held[1]).reshape(T, Hq, D)
    return out


def exact(case, seed):
    if case["op"] == "adjust" and case["B"] * case["rows"] > 20_000:
        return None
    return {"adjust": _exact_adjust, "append": _exact_append, "attend": _exact_attend}[case["op"]](prepare(case, seed))


def work(case):
    c = case
    size = 4 if c["dtype"] == "fp32" else 2
    if c["op"] == "adjust":
        n = c["B"] * c["rows"] * c["V"]
        return {"bytes": 2 * n * size + (n // 8 if c["grammar"] else 0) + 4 * c["B"] * (c["history"] * 3 // 4 + 2 * c["bias"] + c["rows"]), "flops": n}
    B, T, Hkv, D = c["B"], c["T"], c["Hkv"], c["D"]
    if c["op"] == "append":
        n = int(B * T * (0.75 if c["ragged"] else 1)) * Hkv
        # keys and values in, their codes and scales out, the values held out (whole)
        return {"bytes": 2 * n * (D * size + D // 2 + 4) + 2 * B * T * Hkv * D * size + B * T * c["rotary"] * 4, "flops": 2 * n * D * 4 + 3 * n * c["rotary"]}
    L = int(c["L"] * 9 / 16) if c["ragged"] else c["L"]
    return {"bytes": B * (L + T) * Hkv * (D + 8) + 2 * B * T * c["Hq"] * D * size + (B * T * D * 4 if c["rope"] else 0), "flops": 4 * B * T * c["Hq"] * D * (L + T)}
