"""Speculative decoding over a paged key/value cache, with a budget on its slots.

A toy model of one attention layer with random weights stands for the language model, a bigram table for the
draft model.  Each round the draft proposes a few tokens per conversation; the target runs over them at once
(``keops_cache_append``, ``keops_paged_attention`` with the slots' weights accumulated), ``keops_verify_draft``
decides how many stand, and a conversation that outgrows its budget is cut down to it by attention weight
(``keops_cache_evict``).  Lengths stay on the device; the host keeps the page lists.

The weights take up the attention of all drafted rows, before it is known which of them are refused, so a refused
token has a say in what is evicted.  Where that matters, leave ``weights`` out of the call that verifies, and let a
second call over the rows that were accepted accumulate them; it reads the cache once more.

With ``four_bit`` the cache is held in 4 bits and keys and queries turn to their positions in the text on the way
(``keops_cache_append_rotary``; after an eviction a slot's number is no position any more).  With ``rules`` the target's
logits pass ``keops_adjust_logits`` first: repeated tokens are penalised, drafted ones as if they stood, and the upper
half of the vocabulary is forbidden.

    python examples/paged_decode.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import geometric_map_reduce_amd as gm  # noqa: E402


class Pages:
    """The pool and who owns which page."""

    def __init__(self, count, page, heads, dim, dtype, device, four_bit=False):
        self.page = page
        self.scales = {}
        if four_bit:
            self.k, self.v = (torch.zeros((count, page, heads, dim // 2), dtype=torch.uint8, device=device).view(torch.float4_e2m1fn_x2)
                              for _ in range(2))
            self.scales = {name: torch.zeros((count, heads, page, dim // 32), dtype=torch.uint8, device=device).view(torch.float8_e8m0fnu)
                           for name in ("k_scale", "v_scale")}
        else:
            self.k = torch.zeros((count, page, heads, dim), dtype=dtype, device=device)
            self.v = torch.zeros_like(self.k)
        self.weights = torch.zeros((count, heads, page), device=device)
        self.free = list(range(count))

    def take(self, slots):
        n = -(-slots // self.page)
        if n > len(self.free):
            raise RuntimeError("the page pool is exhausted")
        got, self.free = self.free[:n], self.free[n:]
        return got


class Toy:
    """One layer: x = embed(token); attention of 8 query heads over 2 key/value heads; logits = (x + out) @ head."""

    def __init__(self, vocab, dim, seed, device, heads=8, kv_heads=2, dtype=torch.bfloat16):
        g = torch.Generator(device=device).manual_seed(seed)

        def rand(*shape):
            return torch.randn(shape, generator=g, device=device)
        self.heads, self.kv, self.dim, self.dtype = heads, kv_heads, dim, dtype
        width = heads * dim
        self.embed = rand(vocab, width)
        self.wqkv = (rand(width, (heads + 2 * kv_heads) * dim) / width ** 0.5).to(dtype)
        self.head = rand(width, vocab) * 2 / width ** 0.5
        self.bigram = torch.softmax(rand(vocab, vocab) * 2, -1)

    def qkv(self, tokens):
        rows = self.embed[tokens].to(self.dtype) @ self.wqkv
        q, k, v = rows.split([self.heads * self.dim, self.kv * self.dim, self.kv * self.dim], -1)
        # keys and values stay rows of the wide product
        return q.contiguous().view(-1, self.heads, self.dim), k.view(-1, self.kv, self.dim), v.view(-1, self.kv, self.dim)

    def logits(self, tokens, out):
        return (self.embed[tokens] + out.float().flatten(1)) @ self.head


def decode(rounds=40, seqs=6, drafts=3, vocab=199, dim=64, page=16, budget=64, sink=2, recent=16, seed=0, device="cuda", watch=None,
           four_bit=False, rules=False):
    """Runs the loop; returns the generated tokens of every conversation.  ``watch(state)`` sees every round."""
    model = Toy(vocab, dim, seed, device)
    most = budget + drafts + 1
    pages = Pages(2 * (seqs + 1) * -(-most // page), page, model.kv, dim, model.dtype, device, four_bit)
    owned = [pages.take(most) for _ in range(seqs)]
    lens = torch.zeros(seqs, dtype=torch.int32, device=device)
    g = torch.Generator(device=device).manual_seed(seed + 1)
    last = torch.randint(0, vocab, (seqs,), generator=g, device=device)
    text = [[] for _ in range(seqs)]
    step = drafts + 1
    starts = torch.arange(0, seqs * step + 1, step, dtype=torch.int32, device=device)
    counts = torch.full((seqs,), drafts, dtype=torch.int32, device=device)
    freqs = gm.keops_rotary_frequencies(dim, device=device)
    # the texts, with the place of each one's last token, which the target has not seen yet
    said = torch.zeros(seqs, dtype=torch.int32, device=device)
    spoken = torch.zeros((seqs, rounds * step + step), dtype=torch.int32, device=device)
    ahead = torch.arange(step, dtype=torch.int32, device=device)
    penalty = torch.full((seqs,), 1.3, device=device)
    words = -(-vocab // 32)
    allowed = torch.tensor([-1 if 32 * w + 32 <= vocab // 2 else (1 << max(vocab // 2 - 32 * w, 0)) - 1 for w in range(words)],
                           dtype=torch.int32, device=device).repeat(seqs * step, 1)
    for _ in range(rounds):
        table = torch.tensor(owned, dtype=torch.int32, device=device)
        # the draft: each token from the one before it
        token, proposed, draft = last, [], []
        for _ in range(drafts):
            p = model.bigram[token]
            token = torch.multinomial(p, 1, generator=g)[:, 0]
            proposed.append(token)
            draft.append(p)
        proposed, draft = torch.stack(proposed, 1), torch.stack(draft, 1)
        # the target over the last token and the proposed ones
        tokens = torch.cat([last[:, None], proposed], 1).flatten()
        q, k, v = model.qkv(tokens)
        lens += step
        at = said[:, None] + ahead
        if four_bit:
            q = gm.keops_cache_append_rotary(q, k, v, pages.k, pages.v, table, lens, starts, freqs, positions=at.flatten(),
                                             weights=pages.weights, **pages.scales)
        else:
            gm.keops_cache_append(k, v, pages.k, pages.v, table, lens, starts, weights=pages.weights)
        out, lse = gm.keops_paged_attention(q, pages.k, pages.v, table, lens, starts, step, most, weights=pages.weights, decay=1.0,
                                            **pages.scales)
        logits = model.logits(tokens, out)
        if rules:
            spoken.scatter_(1, at.long(), tokens.view(seqs, step).int())
            gm.keops_adjust_logits(logits, starts, tokens=spoken, lens=said + step, repetition=penalty, mask=allowed, out=logits)
        target = torch.softmax(logits, -1).view(seqs, step, vocab)
        kept, accepted = gm.keops_verify_draft(target, draft, proposed.int(), counts,
                                               torch.rand((seqs, drafts), generator=g, device=device),
                                               torch.rand(seqs, generator=g, device=device))
        if watch is not None:
            watch(dict(model=model, pages=pages, table=table, lens=lens.clone(), starts=starts, q=q, k=k, v=v, out=out, lse=lse,
                       tokens=tokens, kept=kept, accepted=accepted))
        # what was refused leaves the cache: its slots are written over
        lens -= drafts - accepted
        said += accepted + 1
        last = kept.gather(1, accepted[:, None].long())[:, 0].long()
        for s, row in enumerate(kept.tolist()):
            text[s] += [t for t in row if t >= 0]
        # one look at the lengths a round decides who is cut: everyone's pages change hands
        if int(lens.max()) + step > most:
            new = [pages.take(most) for _ in range(seqs)]
            _, lens = gm.keops_cache_evict(pages.k, pages.v, pages.weights, table, lens,
                                           torch.tensor(new, dtype=torch.int32, device=device), budget - step, sink=sink, recent=recent,
                                           **pages.scales)
            for old in owned:
                pages.free += old
            owned = new
    return text


if __name__ == "__main__":
    if not torch.cuda.is_available():
        sys.exit("needs a GPU")
    for four_bit in (False, True):
        for s, t in enumerate(decode(four_bit=four_bit, rules=four_bit)):
            print(f"conversation {s}: {len(t)} tokens: {t[:16]} ...")
