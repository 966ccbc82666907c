"""Plain 64-bit forms of the operators around the paged cache (rotary positions, 4-bit blocks, logits), on the CPU,
written from their definitions, with the error bounds of the kernels' arithmetic beside them."""
from __future__ import annotations

import torch

import paged_reference as ref
from paged_reference import U32

LEVELS = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
E2 = torch.float4_e2m1fn_x2


def rotate(x, positions, freqs, interleaved=False, factor=1.0, inverse=False):
    """x [tokens, heads, dim] rotated, in 64 bits."""
    n, x = len(freqs), x.double()
    angle = (positions.double()[:, None] * freqs)[:, None]
    if inverse:
        angle = -angle
    c, s = factor * torch.cos(angle), factor * torch.sin(angle)
    y = x.clone()
    a, b = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., a] * s + x[..., b] * c
    return y


def rotate_bound(x, y, freqs, dtype, factor=1.0):
    """How far the kernel's y may be off: cosine and sine are rounded to 32 bits, two products and a sum to 32 bits,
    each of them at most factor (|a| + |b|), then the result to its type."""
    n, x = len(freqs), x.double().abs()
    if n == 0:
        return torch.zeros_like(y)
    half = torch.finfo(dtype).eps / 2
    size = abs(factor) * (x + torch.cat([x[..., :2 * n].amax(-1, keepdim=True).expand_as(x[..., :2 * n]), x[..., 2 * n:]], -1))
    floor = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}[dtype]
    return half * y.abs() * (1 + 8 * U32) + 4 * U32 * size + floor


def power_top(dtype):
    return 140 if dtype == torch.float16 else 252


def to_4bit(x, dtype):
    """(codes, powers): blocks of 32 columns of x by trying every power from the least on."""
    b = x.double().unflatten(-1, (-1, 32))
    most = b.abs().amax(-1)
    power = torch.zeros(most.shape, dtype=torch.long)
    for p in range(power_top(dtype)):
        # still rounds past 6 under power p: the halfway mark between 6 and 8 belongs to 8
        power = torch.where(most >= 7 * 2.0 ** (p - 127), torch.full_like(power, p + 1), power)
    lost = ~torch.isfinite(b).all(-1)
    y = torch.where(lost[..., None], torch.zeros_like(b), b / torch.exp2(power.double() - 127)[..., None])
    away = (y.abs()[..., None] - LEVELS).abs()
    best = away.amin(-1, keepdim=True)
    tie = (away == best).sum(-1) > 1
    code = away.argmin(-1)                       # of two the lower
    code = torch.where(tie & (code % 2 == 1), code + 1, code) + 8 * torch.signbit(y).long()
    code = code.flatten(-2)
    return (code[..., 0::2] + 16 * code[..., 1::2]).to(torch.uint8), torch.where(lost, torch.full_like(power, 255), power).to(torch.uint8)


def from_4bit(codes, powers):
    """The values in 64 bits."""
    both = torch.cat([LEVELS, -LEVELS])
    x = torch.stack([both[(codes & 15).long()], both[(codes >> 4).long()]], -1).flatten(-2)
    two = torch.where(powers == 255, torch.full(powers.shape, float("nan"), dtype=torch.float64), torch.exp2(powers.double() - 127))
    return x * two.repeat_interleave(32, -1)


class Batch4(ref.Batch):
    """A batch over a cache held in 4 bits: k and v are bytes [pages, page, heads, dim / 2], k_scale and v_scale powers
    [pages, heads, page, dim / 32]."""

    def __init__(self, seed, lens, new, heads, kv_heads, dim, page, dtype=torch.bfloat16, junk=float("nan"), spare=3):
        super().__init__(seed, lens, new, heads, kv_heads, dim, page, dtype, dtype, junk, spare)
        pools = [to_4bit(x, dtype) for x in (self.k, self.v)]
        self.k, self.v = (c for c, _ in pools)
        self.k_scale, self.v_scale = (p.permute(0, 2, 1, 3).contiguous() for _, p in pools)

    def rows(self, pool, scale, s, h, n):
        j = torch.arange(n)
        pi = j // self.page
        there = pi < self.table.shape[1]
        pg = self.table[s, pi.clamp(max=self.table.shape[1] - 1)].long()
        there &= (pg >= 0) & (pg < self.P)
        pg = pg.clamp(0, self.P - 1)
        x = from_4bit(pool[pg, j % self.page, h], scale[pg, h, j % self.page])
        return x.to(self.dtype).double(), there      # read as the nearest values of q's type


def places(b):
    """(token, sequence, slot, page or -1, row) of every token of a batch's sequences."""
    for s, n in enumerate(b.lens):
        a, e = b.starts[s].item(), b.starts[s + 1].item()
        for t in range(a, e):
            j = n - (e - a) + (t - a)
            pg = -1
            if j >= 0 and j // b.page < b.table.shape[1]:
                pg = b.table[s, j // b.page].item()
            yield t, s, j, pg if 0 <= pg < b.P else -1, j % b.page


def append_4bit(b, k, v):
    """Pools and powers of a 4-bit batch after appending k and v (any precision) [tokens, heads, dim]."""
    out = [t.clone() for t in (b.k, b.v, b.k_scale, b.v_scale)]
    kc, vc = to_4bit(k, b.dtype), to_4bit(v, b.dtype)
    for t, _, _, pg, row in places(b):
        if pg >= 0:
            out[0][pg, row], out[1][pg, row] = kc[0][t], vc[0][t]
            out[2][pg, :, row], out[3][pg, :, row] = kc[1][t], vc[1][t]
    return out


def logits(z, starts, text=None, lens=None, prompt=None, rep=None, pres=None, freq=None, ids=None, bias=None, mask=None):
    """In 64 bits; rows of no sequence are NaN."""
    rows, V = z.shape
    out = torch.full((rows, V), float("nan"), dtype=torch.float64)
    for s in range(len(starts) - 1):
        a, e = min(max(int(starts[s]), 0), rows), min(max(int(starts[s + 1]), 0), rows)
        for t in range(a, e):
            y = z[t].double().clone()
            if text is not None:
                end = min(int(lens[s]) - (e - t) + 1, text.shape[1])
                past = [int(x) for x in text[s, :max(end, 0)]]
                for x in {x for x in past if 0 <= x < V}:
                    r = 1.0 if rep is None else rep[s].double()
                    y[x] = y[x] / r if y[x] > 0 else y[x] * r
                    c = sum(1 for i, w in enumerate(past) if w == x and i >= (0 if prompt is None else int(prompt[s])))
                    if c:
                        y[x] -= (0.0 if freq is None else freq[s].double()) * c + (0.0 if pres is None else pres[s].double())
            if ids is not None:
                for x, add in {int(i): v for i, v in zip(ids[s], bias[s].double())}.items():
                    if 0 <= x < V:
                        y[x] += add
            if mask is not None:
                for x in range(V):
                    if not (int(mask[t, x // 32]) >> (x % 32)) & 1:
                        y[x] = -float("inf")
            out[t] = y
    return out
