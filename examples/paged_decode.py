"""Speculative decoding over a paged key/value cache, with a budget on its slots.

A toy model of one attention layer with random weights stands for the language model, a bigram table for the
draft model.  Each round the draft proposes a few tokens per conversation; the target runs over them at once
(``keops_cache_append``, ``keops_paged_attention`` with the slots' weights accumulated), ``keops_verify_draft``
decides how many stand, and a conversation that outgrows its budget is cut down to it by attention weight
(``keops_cache_evict``).  Lengths stay on the device; the host keeps the page lists.

The weights take up the attention of all drafted rows, before it is known which of them are refused, so a refused
token has a say in what is evicted.  Where that matters, leave ``weights`` out of the call that verifies, and let a
second call over the rows that were accepted accumulate them; it reads the cache once more.

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

    def __init__(self, count, page, heads, dim, dtype, device):
        self.page = page
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

    def probabilities(self, tokens, out):
        return torch.softmax((self.embed[tokens] + out.float().flatten(1)) @ self.head, -1)


def decode(rounds=40, seqs=6, drafts=3, vocab=199, dim=64, page=16, budget=64, sink=2, recent=16, seed=0, device="cuda", watch=None):
    """Runs the loop; returns the generated tokens of every conversation.  ``watch(state)`` sees every round."""
    model = Toy(vocab, dim, seed, device)
    most = budget + drafts + 1
    pages = Pages(2 * (seqs + 1) * -(-most // page), page, model.kv, dim, model.dtype, device)
    owned = [pages.take(most) for _ in range(seqs)]
    lens = torch.zeros(seqs, dtype=torch.int32, device=device)
    g = torch.Generator(device=device).manual_seed(seed + 1)
    last = torch.randint(0, vocab, (seqs,), generator=g, device=device)
    text = [[] for _ in range(seqs)]
    step = drafts + 1
    starts = torch.arange(0, seqs * step + 1, step, dtype=torch.int32, device=device)
    counts = torch.full((seqs,), drafts, dtype=torch.int32, device=device)
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
        gm.keops_cache_append(k, v, pages.k, pages.v, table, lens, starts, weights=pages.weights)
        out, lse = gm.keops_paged_attention(q, pages.k, pages.v, table, lens, starts, step, most, weights=pages.weights, decay=1.0)
        target = model.probabilities(tokens, out).view(seqs, step, vocab)
        kept, accepted = gm.keops_verify_draft(target, draft, proposed.int(), counts,
                                               torch.rand((seqs, drafts), generator=g, device=device),
                                               torch.rand(seqs, generator=g, device=device))
        if watch is not None:
            watch(dict(model=model, pages=pages, table=table, lens=lens.clone(), starts=starts, q=q, k=k, v=v, out=out, lse=lse,
                       tokens=tokens, kept=kept, accepted=accepted))
        # what was refused leaves the cache: its slots are written over
        lens -= drafts - accepted
        last = kept.gather(1, accepted[:, None].long())[:, 0].long()
        for s, row in enumerate(kept.tolist()):
            text[s] += [t for t in row if t >= 0]
        # one look at the lengths a round decides who is cut: everyone's pages change hands
        if int(lens.max()) + step > most:
            new = [pages.take(most) for _ in range(seqs)]
            _, lens = gm.keops_cache_evict(pages.k, pages.v, pages.weights, table, lens,
                                           torch.tensor(new, dtype=torch.int32, device=device), budget - step, sink=sink, recent=recent)
            for old in owned:
                pages.free += old
            owned = new
    return text


if __name__ == "__main__":
    if not torch.cuda.is_available():
        sys.exit("needs a GPU")
    for s, t in enumerate(decode()):
        print(f"conversation {s}: {len(t)} tokens: {t[:16]} ...")
