"""One speculative decoding loop, every step of it in the library's kernels but the matrix products.

A toy two-layer model (random weights) decodes a batch greedily: prompt-lookup drafts from the
history (spec_ngram_draft), the drafts' keys and values into the 4-bit paged cache with their
rotation (spec_kv_append), their attention over it (spec_kv_attention), a repetition penalty and
a mask of allowed tokens on the logits (spec_logit_adjust), and the verification
(spec_verify_greedy).  A rejected draft needs no clean-up: the next step's tokens are appended
over its slots.

    python examples/verify_step.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import speculative_decoding_verify_spec_gb300 as sv  # noqa: E402


class Model:
    """Two layers of grouped-query attention over the paged cache, and an output head."""

    def __init__(self, vocab=256, heads=8, kv_heads=2, head_dim=64, layers=2, max_len=512, batch=4, page=16, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        width = heads * head_dim
        rand = lambda *s: (torch.randn(s, generator=g, device="cuda") * s[0] ** -0.5).to(torch.bfloat16)  # noqa: E731
        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, head_dim
        self.embedding, self.head = rand(vocab, width) * 16, rand(width, vocab)
        self.layers = [(rand(width, (heads + 2 * kv_heads) * head_dim), rand(width, width)) for _ in range(layers)]
        angle = torch.arange(max_len, device="cuda")[:, None] * 10000.0 ** (-torch.arange(head_dim // 2, device="cuda") / (head_dim // 2))
        self.cos, self.sin = angle.cos(), angle.sin()
        pages = max_len // page
        self.table = torch.randperm(batch * pages, generator=g, device="cuda").to(torch.int32).reshape(batch, pages)
        size = sv.spec_kv_page_bytes(page, head_dim)
        self.caches = [torch.empty((batch * pages, kv_heads, size), dtype=torch.uint8, device="cuda") for _ in range(layers)]

    def __call__(self, tokens, start):
        """Logits [B, T, vocab] of tokens [B, T] that follow `start` [B] cached ones."""
        x = self.embedding[tokens.long()]
        q, k = self.heads * self.head_dim, self.kv_heads * self.head_dim
        rotation = dict(cos=self.cos, sin=self.sin)
        for (w_in, w_out), cache in zip(self.layers, self.caches):
            qkv = (x @ w_in).split([q, k, k], -1)
            qh, kh, vh = (t.unflatten(-1, (-1, self.head_dim)) for t in qkv)
            sv.spec_kv_append(kh, vh, cache, self.table, start, **rotation)
            x = x + sv.spec_kv_attention(qh, cache, self.table, start, **rotation).flatten(-2) @ w_out
        return x @ self.head


def decode(model, prompt, steps, gamma, repetition=1.2, allowed_words=None):
    """Decodes `steps` verified steps after prompt [B, n] int32; returns (history [B, max], lengths [B])."""
    B, n = prompt.shape
    dev = prompt.device
    history = torch.zeros((B, n + steps * (gamma + 1)), dtype=torch.int32, device=dev)
    history[:, :n] = prompt
    lengths = torch.full((B,), n, dtype=torch.int32, device=dev)
    penalty = torch.full((B,), repetition, device=dev)
    allowed = None if allowed_words is None else allowed_words.expand(B, gamma + 1, -1).contiguous()
    model(prompt[:, :-1].contiguous(), torch.zeros_like(lengths))  # the last token's turn comes with the drafts
    column = torch.arange(gamma + 1, device=dev)
    for _ in range(steps):
        last = history.gather(1, lengths[:, None].long() - 1)
        if gamma:
            drafts, _ = sv.spec_ngram_draft(history, lengths, 2, gamma, True)
        else:
            drafts = torch.empty((B, 0), dtype=torch.int32, device=dev)
        logits = model(torch.cat([last, drafts], 1), lengths - 1)
        sv.spec_logit_adjust(logits, history=history, lengths=lengths, draft_tokens=drafts, repetition=penalty, allowed=allowed, out=logits)
        accepted, tokens = sv.spec_verify_greedy(logits, drafts)
        at = (lengths[:, None] + column).long()
        keep = column <= accepted[:, None]
        history.scatter_(1, at, torch.where(keep, tokens, history.gather(1, at)))
        lengths = lengths + accepted + 1
    return history, lengths


def main():
    model = Model()
    prompt = torch.arange(12, dtype=torch.int32, device="cuda").repeat(4, 2) + 7 * torch.arange(4, dtype=torch.int32, device="cuda")[:, None]
    history, lengths = decode(model, prompt, steps=20, gamma=4)
    for row, n in zip(history.tolist(), lengths.tolist()):
        print(n, "tokens:", row[:n])


if __name__ == "__main__":
    main()
