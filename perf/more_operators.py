"""The paged cache held in 8 bits: what its operators compute, on real sizes.

Three operators, each in a plain form (elementary torch operations) and as the call that a
user of the package makes:

  append   the new tokens' keys (rotated) and values into a paged cache held in 8 bits, with a
           scale for each block of 16 tokens and head; gives back the values held for the new
           tokens, and the cache
  read     tokens of the cache back in 16 bits: a range of them, or listed ones
  attend   the new tokens' attention (chain or tree) over that cache

The cache is [pages][heads][page_size * (2 D + 1)] bytes.  Per page and head: the keys' codes, the
values' codes, then 16 bytes for each block of 16 slots.  A code is a float of 8 bits (4 of exponent, 3 of
mantissa, largest 448).  Code d of slot t is at byte t // 8 * 8 D + d // 16 * 128 + t % 8 * 16 + d % 16.  A block's
bytes are one 32-bit word for its keys and one for its values, and 8 unused bytes; a word's upper half is the
block's scale as a bfloat16, its lower half has bit t % 16 set if slot t's vector had a NaN or an infinity.

A block's scale is a power of two: with A the largest magnitude among the vectors written into the block, 2^(e - 8)
where 2^e is the least power of two that is not below A, within 2^-40 .. 2^40; and no less than what it was if the
block holds tokens from before, whose codes are then rounded to the new scale.  A number x is held as the
code nearest to x / scale (ties to even, zero as +0), and stands for code * scale.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------------------- cases


def listed():
    return [
        # one sequence decoding one token, into a block that holds twelve tokens
        dict(name="append_one", op="append", B=1, T=1, Hkv=8, D=128, dtype="bf16", page=16, L=700, rotary=128, interleaved=False, ragged=False),
        # eight drafts and the last token of a full batch, across the borders of blocks
        dict(name="append_chain", op="append", B=256, T=9, Hkv=8, D=128, dtype="bf16", page=64, L=509, rotary=128, interleaved=False, ragged=True),
        # prompts of odd lengths taken in at once, a rotation over part of the head in neighbouring pairs
        dict(name="append_prompts", op="append", B=8, T=2001, Hkv=16, D=64, dtype="fp16", page=32, L=100, rotary=32, interleaved=True, ragged=True),
        # one long prompt, wide heads
        dict(name="append_long", op="append", B=1, T=16384, Hkv=4, D=256, dtype="bf16", page=128, L=0, rotary=256, interleaved=False, ragged=False),
        # the accepted path of a token tree, to be appended again behind the context
        dict(name="read_path", op="read", B=64, T=7, Hkv=8, D=128, dtype="bf16", page=64, L=1000, listed=True, ragged=True),
        # a shared prefix handed to an attention in 16 bits
        dict(name="read_prefix", op="read", B=4, T=20001, Hkv=8, D=128, dtype="bf16", page=64, L=0, listed=False, ragged=False),
        # one sequence decoding one token
        dict(name="attend_one", op="attend", B=1, T=1, Hq=32, Hkv=8, D=128, dtype="bf16", page=16, L=700, tree=False, rope=True, ragged=False),
        # verifying eight drafts of a batch with contexts of all lengths
        dict(name="attend_drafts", op="attend", B=64, T=9, Hq=32, Hkv=8, D=128, dtype="bf16", page=64, L=4096, tree=False, rope=True, ragged=True),
        # verifying a token tree of 64 nodes
        dict(name="attend_nodes", op="attend", B=64, T=64, Hq=16, Hkv=4, D=64, dtype="fp16", page=32, L=2047, tree=True, rope=False, ragged=True),
        # a large batch decoding single tokens over long contexts
        dict(name="attend_batch", op="attend", B=256, T=1, Hq=64, Hkv=8, D=128, dtype="bf16", page=64, L=8192, tree=False, rope=True, ragged=True),
        # five drafts over one very long context, wide heads
        dict(name="attend_context", op="attend", B=1, T=6, Hq=16, Hkv=4, D=256, dtype="bf16", page=128, L=200001, tree=False, rope=True, ragged=False),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "read", "attend"])
    D = rng.choice([64, 128, 256])
    Hkv = rng.choice([1, 2, 4, 5, 8, 16])
    page, dtype = rng.choice([16, 32, 48, 64, 128]), rng.choice(["bf16", "fp16"])
    if op == "append":
        B, T, L = _logint(rng, 1, 256), _logint(rng, 1, 16384), rng.choice([0, _logint(rng, 1, 1000)])
        while B * T * Hkv * D > 16_500_000:
            T = max(1, T // 2)
            B = B if T > 1 else max(1, B // 2)
        return dict(op=op, B=B, T=T, Hkv=Hkv, D=D, dtype=dtype, page=page, L=L, rotary=rng.choice([D, D, D // 2, 0]),
                    interleaved=rng.random() < 0.4, ragged=rng.random() < 0.5)
    if op == "read":
        few = rng.random() < 0.5
        B, T, L = _logint(rng, 1, 256), rng.randint(1, 17) if few else _logint(rng, 16, 20000), _logint(rng, 1, 1000)
        while B * (T + L) * Hkv * D > 80_000_000:
            B, T = (B // 2, T) if B > 4 else (B, max(1, T // 2))
        return dict(op=op, B=B, T=T, Hkv=Hkv, D=D, dtype=dtype, page=page, L=L, listed=few, ragged=rng.random() < 0.5)
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


def prepare(case, seed):
    c, dev = case, "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    B, T, Hkv, D, page, L = c["B"], c["T"], c["Hkv"], c["D"], c["page"], c["L"]
    dt = DT[c["dtype"]]
    s = dict(case=c)
    start = torch.randint(L // 8, L + 1, (B,), generator=host) if c["ragged"] else torch.full((B,), L)
    some = c["op"] != "attend" and c["ragged"]
    s["count"] = torch.randint((T + 1) // 2, T + 1, (B,), generator=host).to(dev, torch.int32) if some else None
    width = (L + T + page - 1) // page
    pages = B * width + 3
    s["page_table"] = torch.randperm(pages, generator=host)[:B * width].reshape(B, width).to(dev, torch.int32)
    s["start"] = start.to(dev, torch.int32)
    rotary = c["rotary"] if c["op"] == "append" else D if c["op"] == "attend" and c["rope"] else 0
    s["cos"], s["sin"] = _tables(L + T, rotary) if rotary else (None, None)
    # keys have a few strong channels
    strong = 4 * torch.randn((Hkv, D), device=dev, generator=gen) * (torch.rand((Hkv, D), device=dev, generator=gen) < 0.04)
    if c["op"] == "append":
        s["k"] = (torch.randn((B, T, Hkv, D), device=dev, generator=gen) + strong).to(dt)
        s["v"] = torch.randn((B, T, Hkv, D), device=dev, generator=gen).to(dt)
    s["slots"] = None
    if c["op"] == "read" and c["listed"]:  # a path: the root's slot, then some behind it
        hop = torch.randint(1, 4, (B, T), generator=host).cumsum(1) - 1
        s["slots"] = torch.minimum(start[:, None] + hop, torch.tensor(L + T - 1)).to(dev, torch.int32)
    s["positions"], s["parent"] = None, None
    if c["op"] == "attend":
        s["q"] = torch.randn((B, T, c["Hq"], D), device=dev, generator=gen).to(dt)
        if c["tree"]:
            s["parent"] = _parents(T, host).to(dev)
            depth = _ancestors(s["parent"]).sum(1) - 1
            s["positions"] = (s["start"][:, None] + depth[None, :]).to(torch.int32)
    # the whole pool is filled, a part at a time: pages that no sequence reads hold old tokens
    s["cache"] = torch.empty((pages, Hkv, page * (2 * D + 1)), dtype=torch.uint8, device=dev)
    step = max(1, 400_000_000 // (Hkv * page * D * 8))
    for p in range(0, pages, step):
        n = min(step, pages - p)
        loud = _power(torch.randint(-2, 3, (n, 1, page // 16, 1, 1), device=dev, generator=gen)).float()  # texts differ in loudness
        k = (torch.randn((n, Hkv, page // 16, 16, D), device=dev, generator=gen) + strong[:, None, None]) * loud
        v = torch.randn((n, Hkv, page // 16, 16, D), device=dev, generator=gen) * loud
        parts, words = [], []
        for x in (k, v):
            scale = _scale(x.abs().amax((-1, -2)))
            code = (x / scale[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
            code = torch.where(code == 128, 0, code).reshape(n, Hkv, page // 8, 8, D // 16, 16)
            parts.append(code.transpose(3, 4).reshape(n, Hkv, page * D))
            words.append(_word(scale, 0))
        words += [torch.zeros_like(words[0])] * 2
        parts.append(torch.stack(words, -1).reshape(n, Hkv, -1).view(torch.uint8))
        s["cache"][p:p + n] = torch.cat(parts, -1)
    return s


# ------------------------------------------------------------------------- plain forms


def _power(e):
    """2 ** e in 64 bits, of whole numbers: by their bits, for a power or an ldexp on the GPU need not be exact."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _scale(largest):
    """The scale of blocks whose largest magnitudes are these, in their type."""
    m, e = torch.frexp(largest)  # m in 1/2 .. 1
    e = torch.where(m == 0.5, e - 1, e) - 8
    return _power(torch.where(largest > 0, e, -40).clamp(-40, 40)).to(largest.dtype)


def _word(scale, bad):
    """Words (int32) of scales and of the bad vectors' bits."""
    return scale.to(torch.bfloat16).view(torch.int16).to(torch.int32) << 16 | bad


def _code(y):
    """Codes (uint8) nearest to y, float64 of at most 448."""
    m, e = torch.frexp(y.abs())
    e = (e - 1).clamp(min=-6)
    n = (y.abs() * _power(3 - e)).round()  # 8 .. 16, or less at the lowest exponent
    code = torch.where(n >= 8, (e + 6) * 8 + n, n).to(torch.uint8)  # (16: the next exponent's first)
    return torch.where((y < 0) & (code > 0), code + 128, code)


def _number(code):
    """What codes stand for, in 32 bits."""
    return code.view(torch.float8_e4m3fn).float()


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


def _append(s):
    c = s["case"]
    B, T, Hkv, D, page = c["B"], c["T"], c["Hkv"], c["D"], c["page"]
    dev, dt, cache = s["k"].device, s["k"].dtype, s["cache"]
    start, t = s["start"].long()[:, None], torch.arange(T, device=dev)
    count = s["count"].long()[:, None] if s["count"] is not None else torch.full((B, 1), T, device=dev)
    # the blocks that the new tokens touch, token by token: which sequence, which slot, kept or new
    first = start // 16 * 16
    slot = first + torch.arange((T + 30) // 16 * 16, device=dev)
    touched = (slot // 16 * 16 < start + count).reshape(B, -1, 16)[..., 0] & (count > 0)
    b, j = touched.nonzero(as_tuple=True)  # blocks
    slot = (first[b, 0] + 16 * j)[:, None] + torch.arange(16, device=dev)  # [n, 16]
    kept, new = slot < start[b], (slot >= start[b]) & (slot < (start + count)[b])
    pg = s["page_table"].long()[b, slot[:, 0] // page]
    src = b[:, None] * T + (slot - start[b]).clamp(0, T - 1)
    dims, head = torch.arange(D, device=dev), torch.arange(Hkv, device=dev)
    tok = slot % page
    byte = (tok // 8 * 8 * D + tok % 8 * 16)[:, :, None, None] + (dims // 16 * 128 + dims % 16)
    word = 2 * page * D + tok[:, 0] // 16 * 16
    out = []
    # codes near a border between two need more than 32 bits
    for i, x in enumerate((_rotate(s["k"].double(), s["cos"], s["sin"], start + t, c["interleaved"]), s["v"].double())):
        x = x.reshape(B * T, Hkv, D)[src]  # [n, 16, Hkv, D]
        scale = _scale(torch.where(new[..., None, None], x.abs(), 0.0).amax((1, 3)))  # [n, Hkv]
        at = (word + 4 * i)[:, None, None] + torch.arange(4, device=dev)
        old = (cache[pg[:, None, None], head[:, None], at].view(torch.int32)[..., 0] >> 16 << 16).view(torch.float32).double()
        scale = torch.where(kept.any(1)[:, None], torch.maximum(scale, old), scale)
        where = pg[:, None, None, None], head[:, None], byte + i * page * D
        was = cache[where]
        y = torch.where(kept[..., None, None], _number(was).double() * old[:, None, :, None], x)
        code = torch.where((kept | new)[..., None, None], _code(y / scale[:, None, :, None]), was)
        cache[where] = code
        cache[pg[:, None, None], head[:, None], at] = _word(scale, 0)[..., None].view(torch.uint8)
        held = torch.zeros((B * T, Hkv, D), dtype=dt, device=dev)
        held[src[new]] = (_number(code).double() * scale[:, None, :, None])[new].to(dt)
        out.append(held.reshape(B, T, Hkv, D))
    return out[0], out[1], cache


def _unpack(pages, page, D):
    """Keys and values [n, H, page, D] in 32 bits that page bytes [n, H, page * (2 D + 1)] stand for."""
    n, H = pages.shape[:2]
    word = pages[..., 2 * page * D:].contiguous().view(torch.int32).reshape(n, H, page // 16, 4)
    out = []
    for i in (0, 1):
        x = _number(pages[..., i * page * D:(i + 1) * page * D].contiguous()).reshape(n, H, page // 8, D // 16, 8, 16)
        scale = (word[..., i] >> 16 << 16).view(torch.float32)
        out.append(x.transpose(3, 4).reshape(n, H, page, D) * scale.repeat_interleave(16, -1)[..., None])
    return out


def _read(s):
    c = s["case"]
    B, T, D, page = c["B"], c["T"], c["D"], c["page"]
    dev, dt, cache = s["cache"].device, DT[c["dtype"]], s["cache"]
    t = torch.arange(T, device=dev)
    slot = s["slots"].long() if s["slots"] is not None else s["start"].long()[:, None] + t
    pg = s["page_table"].long().gather(1, slot // page)[..., None, None]
    tok, dims, head = (slot % page)[..., None, None], torch.arange(D, device=dev), torch.arange(c["Hkv"], device=dev)[:, None]
    live = (t < s["count"][:, None])[..., None, None] if s["count"] is not None else torch.ones((B, T, 1, 1), dtype=torch.bool, device=dev)
    out = []
    for i in (0, 1):
        code = cache[pg, head, i * page * D + tok // 8 * 8 * D + dims // 16 * 128 + tok % 8 * 16 + dims % 16]
        word = cache[pg, head, 2 * page * D + tok // 16 * 16 + 4 * i + torch.arange(4, device=dev)].view(torch.int32)
        out.append(torch.where(live, _number(code) * (word >> 16 << 16).view(torch.float32), 0.0).to(dt))
    return out[0], out[1]


def _attend(s):
    c = s["case"]
    B, T, Hq, Hkv, D, page = c["B"], c["T"], c["Hq"], c["Hkv"], c["D"], c["page"]
    dev, dt = s["q"].device, s["q"].dtype
    at = s["positions"] if s["positions"] is not None else s["start"][:, None] + torch.arange(T, device=dev)
    q = _rotate(s["q"].float(), s["cos"], s["sin"], at, False).reshape(B, T, Hkv, Hq // Hkv, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D)
    width = s["page_table"].shape[1]
    k, v = _unpack(s["cache"][s["page_table"].flatten().long()], page, D)
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
        return _append(s) if op == "append" else _read(s) if op == "read" else _attend(s)
    import speculative_decoding_verify_spec_gb300 as sv
    if op == "append":
        k, v = sv.spec_kv8_append(s["k"], s["v"], s["cache"], s["page_table"], s["start"], new_lens=s["count"], cos=s["cos"],
                                  sin=s["sin"], interleaved=s["case"]["interleaved"], return_values=True)
        return k, v, s["cache"]
    if op == "read":
        return sv.spec_kv8_read(s["cache"], s["page_table"], s["start"], s["case"]["T"], lens=s["count"], slots=s["slots"],
                                dtype=DT[s["case"]["dtype"]])
    return sv.spec_kv8_attention(s["q"], s["cache"], s["page_table"], s["start"], parent=s["parent"], cos=s["cos"], sin=s["sin"],
                                 positions=s["positions"])


# ---------------------------------------------------------------- in 64 bits, and costs


_TWOS = [2.0**n for n in range(-64, 65)]
_EIGHT = [(-1) ** (n >> 7) * ((n & 7) * 2.0**-9 if n & 120 == 0 else (8 + (n & 7)) * 2.0 ** ((n >> 3 & 15) - 10)) for n in range(256)]


def _exact_held(s, b, n):
    """Keys and values [n, H, D] of sequence b's first n slots."""
    c = s["case"]
    D, page, dev = c["D"], c["page"], s["cache"].device
    rows = s["cache"][s["page_table"][b, :(n + page - 1) // page].long()]
    number, twos = (torch.tensor(x, dtype=torch.float64, device=dev) for x in (_EIGHT, _TWOS))
    t, d = torch.arange(n, device=dev)[:, None], torch.arange(D, device=dev)
    pg, tok = t // page, t % page
    out = []
    for i in (0, 1):
        code = rows[pg, :, i * page * D + tok // 8 * (8 * D) + tok % 8 * 16 + d // 16 * 128 + d % 16]  # [n, D, H]
        at = 2 * page * D + tok // 16 * 16 + 4 * i
        high = rows[pg, :, at + 3].long() * 2 + rows[pg, :, at + 2].long() // 128 - 127  # the scale's exponent
        out.append((number[code.long()] * twos[high + 64]).transpose(1, 2))
    return out


def _exact_append(s):
    c = s["case"]
    B, T, L = c["B"], c["T"], c["L"]
    k, v = s["k"].double().clone(), s["v"].double()
    at = s["start"][:, None].long() + torch.arange(T, device="cuda")
    for i in range(0 if s["cos"] is None else s["cos"].shape[1]):
        a, b = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + s["cos"].shape[1])
        turn = torch.complex(s["cos"][at, i].double(), s["sin"][at, i].double())[..., None]
        z = torch.complex(k[..., a], k[..., b]) * turn
        k[..., a], k[..., b] = z.real, z.imag
    number, twos = (torch.tensor(x, dtype=torch.float64, device="cuda") for x in (_EIGHT[:127], _TWOS))
    middle = (number[1:] + number[:-1]) / 2
    held = [torch.zeros_like(v), torch.zeros_like(v)]
    words = s["cache"][:, :, 2 * c["page"] * c["D"]:].reshape(s["cache"].shape[0], c["Hkv"], -1, 4, 4)
    starts, counts = s["start"].tolist(), [T] * B if s["count"] is None else s["count"].tolist()
    for b in range(B):
        for first in range(starts[b] // 16 * 16, starts[b] + counts[b], 16):
            lo, hi = max(first - starts[b], 0), min(first + 16 - starts[b], counts[b])
            for i, x in enumerate((k, v)):
                x = x[b, lo:hi]
                # the first power of two, times 256, that is not below the largest magnitude
                scale = twos[torch.bucketize(x.abs().amax((0, 2)), 256 * twos).clamp(24, 104)]
                if first < starts[b]:
                    pg = int(s["page_table"][b, first // c["page"]])
                    w = words[pg, :, first % c["page"] // 16, i].long()
                    scale = torch.maximum(scale, twos[w[:, 3] * 2 + w[:, 2] // 128 - 127 + 64])
                y = x / scale[:, None]
                up = torch.bucketize(y.abs(), middle, right=True)  # a tie goes up, and back where that is odd
                tie = (up > 0) & (y.abs() == middle[(up - 1).clamp(min=0)]) & (up % 2 == 1)
                held[i][b, lo:hi] = torch.copysign(number[up - tie.long()], y) * scale[:, None]
    return held[0], held[1], None


def _exact_read(s):
    c = s["case"]
    B, T = c["B"], c["T"]
    out = torch.zeros((2, B, T, c["Hkv"], c["D"]), dtype=torch.float64, device="cuda")
    for b in range(B):
        n = T if s["count"] is None else int(s["count"][b])
        slot = s["slots"][b, :n].long() if s["slots"] is not None else int(s["start"][b]) + torch.arange(n, device="cuda")
        k, v = _exact_held(s, b, int(slot.max()) + 1)
        out[0, b, :n], out[1, b, :n] = k[slot], v[slot]
    return out[0], out[1]


def _exact_attend(s):
    c = s["case"]
    B, T, Hq, Hkv, D = c["B"], c["T"], c["Hq"], c["Hkv"], c["D"]
    start, up = s["start"].tolist(), s["parent"].tolist() if c["tree"] else [i - 1 for i in range(T)]
    lines = torch.zeros((T, T), dtype=torch.bool, device="cuda")
    for i in range(T):
        if i:
            lines[i] = lines[up[i]]
        lines[i, i] = True
    out = torch.empty((B, T, Hq, D), dtype=torch.float64, device="cuda")
    for b in range(B):
        k, v = _exact_held(s, b, start[b] + T)
        q = s["q"][b].double()
        if s["cos"] is not None:
            at = (s["positions"][b] if s["positions"] is not None else start[b] + torch.arange(T, device="cuda")).long()
            z = torch.complex(q[..., :D // 2], q[..., D // 2:]) * torch.complex(s["cos"][at].double(), s["sin"][at].double())[:, None]
            q = torch.cat([z.real, z.imag], -1)
        x = torch.einsum("thgd,nhd->htgn", q.reshape(T, Hkv, Hq // Hkv, D), k) / math.sqrt(D)
        x[..., start[b]:].masked_fill_(~lines[None, :, None], -math.inf)
        out[b] = torch.einsum("htgn,nhd->thgd", torch.softmax(x, -1), v).reshape(T, Hq, D)
    return out


def exact(case, seed):
    if case["op"] == "append" and case["B"] * case["T"] > 60_000:
        return None
    return {"append": _exact_append, "read": _exact_read, "attend": _exact_attend}[case["op"]](prepare(case, seed))


def work(case):
    c = case
    B, T, Hkv, D = c["B"], c["T"], c["Hkv"], c["D"]
    if c["op"] == "append":
        n = int(B * T * (0.75 if c["ragged"] else 1)) * Hkv
        # keys and values in, their codes and the blocks' words out, the values held out (whole)
        return {"bytes": 2 * n * (2 * D + D) + n + 2 * B * T * Hkv * D * 2 + B * T * c["rotary"] * 4, "flops": 2 * n * D * 2 + 3 * n * c["rotary"]}
    if c["op"] == "read":
        n = int(B * T * (0.75 if c["ragged"] else 1)) * Hkv
        return {"bytes": n * (2 * D + (8 if c["listed"] else 1)) + 2 * B * T * Hkv * D * 2, "flops": 2 * n * D}
    L = int(c["L"] * 9 / 16) if c["ragged"] else c["L"]
    return {"bytes": B * (L + T) * Hkv * (2 * D + 1) + 2 * B * T * c["Hq"] * D * 2 + (B * T * D * 4 if c["rope"] else 0), "flops": 4 * B * T * c["Hq"] * D * (L + T)}
