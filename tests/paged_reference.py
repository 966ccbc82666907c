"""Plain 64-bit forms of the paged cache operators and of draft verification, on the CPU, written
from their definitions, with the error bounds of the kernels' arithmetic beside them."""
from __future__ import annotations

import math

import torch

U32 = 2.0 ** -24        # half a step of fp32


class Batch:
    """A paged cache and a batch of sequences over it, as CPU tensors.

    lens, new: slots and new tokens of every sequence.  Pages are dealt in a shuffled order; rows that
    no sequence uses hold `junk`.  dtype: q's type; cache: the pool's."""

    def __init__(self, seed, lens, new, heads, kv_heads, dim, page, dtype=torch.bfloat16, cache=None, junk=float("nan"),
                 spare=3):
        g = torch.Generator().manual_seed(seed)
        self.gen = g
        self.lens, self.new = list(lens), list(new)
        self.heads, self.kv, self.dim, self.page = heads, kv_heads, dim, page
        self.dtype, self.cache = dtype, cache or dtype
        self.window, self.scale = 0, 1.0 / math.sqrt(dim)
        S = len(lens)
        used = [-(-n // page) for n in lens]
        P = sum(used) + spare
        self.P = P
        order = torch.randperm(P, generator=g).to(torch.int32)
        width = max(used + [1])
        self.table = torch.full((S, width), -1, dtype=torch.int32)
        at = 0
        for s, u in enumerate(used):
            self.table[s, :u] = order[at:at + u]
            at += u
        self.free = order[at:]
        self.k_scale = self.v_scale = None
        if self.cache.itemsize == 1:
            self.k_scale = 0.01 + 0.01 * torch.rand(kv_heads, generator=g)
            self.v_scale = 0.01 + 0.01 * torch.rand(kv_heads, generator=g)
        self.k = self._pool(self.k_scale, junk)
        self.v = self._pool(self.v_scale, junk)
        starts = [0]
        for m in new:
            starts.append(starts[-1] + m)
        self.starts = torch.tensor(starts, dtype=torch.int32)
        self.T = starts[-1]
        self.q = (torch.randn((self.T, heads, dim), generator=g) * 2).to(dtype)
        self.weights = None

    def _pool(self, scale, junk):
        full = torch.full((self.P, self.page, self.kv, self.dim), junk)
        for s, n in enumerate(self.lens):
            for j0 in range(0, n, self.page):
                rows = min(self.page, n - j0)
                x = torch.randn((rows, self.kv, self.dim), generator=self.gen)
                if scale is not None:
                    x = (x / scale[:, None]).clamp(-448, 448)
                full[self.table[s, j0 // self.page].item(), :rows] = x
        return full.to(self.cache)

    def lens_t(self):
        return torch.tensor(self.lens, dtype=torch.int32)

    def rows(self, pool, scale, s, h, n):
        """Slots 0 .. n-1 of sequence s, head h in 64 bits, and which are there."""
        j = torch.arange(n)
        pi = j // self.page
        there = pi < self.table.shape[1]
        pg = self.table[s, pi.clamp(max=self.table.shape[1] - 1)].long()
        there &= (pg >= 0) & (pg < self.P)
        x = pool[pg.clamp(0, self.P - 1), j % self.page, h].to(torch.float64)
        return (x if scale is None else x * scale[h].double()), there


def attention(b: Batch, decay=0.0):
    """out, lse, weights and bounds of the kernel's error for each."""
    T, Hq, D, G = b.T, b.heads, b.dim, b.heads // b.kv
    out = torch.zeros((T, Hq, D), dtype=torch.float64)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64)
    tol, lse_tol = torch.zeros_like(out), torch.zeros_like(lse)
    w = None if b.weights is None else b.weights.double().clone()
    w_tol = None if w is None else torch.zeros_like(w)
    half = torch.finfo(b.dtype).eps / 2
    for s, n in enumerate(b.lens):
        a, e = b.starts[s].item(), b.starts[s + 1].item()
        if n == 0:
            continue
        for h in range(b.kv):
            k, there = b.rows(b.k, b.k_scale, s, h, n)
            v, _ = b.rows(b.v, b.v_scale, s, h, n)
            mass, mass_tol = torch.zeros(n, dtype=torch.float64), torch.zeros(n, dtype=torch.float64)
            for t in range(a, e):
                pos = n - (e - a) + (t - a)
                j = torch.arange(n)
                sees = there & (j <= pos)
                if b.window:
                    sees &= j > pos - b.window
                at = torch.nonzero(sees)[:, 0]
                for g in range(G):
                    x = b.q[t, h * G + g].double()
                    if len(at) == 0:
                        continue
                    z = (k[at] @ x) * b.scale
                    # fp32 sums of D exact products, the scale's and the exponent's roundings
                    dz = ((k[at].abs() @ x.abs()) * abs(b.scale) * (D + 8) * U32 + 8 * U32 * z.abs()).max().item()
                    L = torch.logsumexp(z, 0)
                    p = torch.exp(z - L)
                    out[t, h * G + g] = p @ v[at]
                    lse[t, h * G + g] = L
                    A = p @ v[at].abs()
                    c = 2 * dz + (len(at) + 64) * U32
                    # p and out are rounded to 16 bits; p of fp16 has an absolute floor of 2^-25
                    floor = 2.0 ** -25 * v[at].abs().sum(0) if b.dtype == torch.float16 else 0.0
                    tol[t, h * G + g] = half * (out[t, h * G + g].abs() + A) * (1 + half) + c * A + floor + \
                        (2.0 ** -25 if b.dtype == torch.float16 else 0.0)
                    lse_tol[t, h * G + g] = dz + (len(at) + 64) * U32 + 16 * U32 * (1 + abs(L.item()))
                    mass[at] += p
                    mass_tol[at] += p * (2 * dz + (len(at) + 64) * U32 + 48 * U32 * (1 + abs(L.item())))
            if w is not None:
                jj = torch.nonzero(there)[:, 0]
                pg, row = b.table[s, jj // b.page].long(), jj % b.page
                old = b.weights[pg, h, row].double()
                w[pg, h, row] = (decay * old if decay else 0.0) + mass[jj]
                w_tol[pg, h, row] = mass_tol[jj] + (e - a) * G * U32 * mass[jj] + \
                    (4 * U32 * (decay * old).abs() if decay else 0.0) + 1e-37
    return out, lse, w, tol, lse_tol, w_tol


def append(b: Batch, k, v):
    """The pools, and the weights, after appending k and v [tokens, heads, dim]."""
    kp, vp = b.k.clone(), b.v.clone()
    w = None if b.weights is None else b.weights.clone()

    def held(x, scale, h):
        if scale is None:
            return x.to(b.cache)
        return (x.float() / scale[h]).clamp(-448, 448).to(b.cache)

    for s, n in enumerate(b.lens):
        a, e = b.starts[s].item(), b.starts[s + 1].item()
        for t in range(a, e):
            j = n - (e - a) + (t - a)
            if j < 0 or j // b.page >= b.table.shape[1]:
                continue
            pg = b.table[s, j // b.page].item()
            if not 0 <= pg < b.P:
                continue
            for h in range(b.kv):
                kp.view(torch.uint8)[pg, j % b.page, h] = held(k[t, h], b.k_scale, h).view(torch.uint8)
                vp.view(torch.uint8)[pg, j % b.page, h] = held(v[t, h], b.v_scale, h).view(torch.uint8)
                if w is not None:
                    w[pg, h, j % b.page] = 0.0
    return kp, vp, w


def evict(b: Batch, new_table, budget, sink, recent):
    S, H = len(b.lens), b.kv
    kept = torch.full((S, H, budget), -1, dtype=torch.int32)
    lens = torch.tensor([min(n, budget) for n in b.lens], dtype=torch.int32)
    kp, vp, w = b.k.clone(), b.v.clone(), b.weights.clone()
    for s, n in enumerate(b.lens):
        for h in range(H):
            if n <= budget:
                keep = list(range(n))
            else:
                def rank(j):
                    pg = b.table[s, j // b.page].item()
                    x = b.weights[pg, h, j % b.page].item() if 0 <= pg < b.P else None
                    if x is None:
                        return (2, 0.0, j)
                    if x != x:
                        return (0, 0.0, j)
                    return (1, -x, j)
                middle = sorted(range(sink, n - recent), key=rank)[:budget - sink - recent]
                keep = list(range(sink)) + sorted(middle) + list(range(n - recent, n))
            kept[s, h, :len(keep)] = torch.tensor(keep, dtype=torch.int32)
            for r, j in enumerate(keep):
                pg, to = b.table[s, j // b.page].item(), new_table[s, r // b.page].item()
                if not (0 <= pg < b.P and 0 <= to < b.P):
                    continue
                kp.view(torch.uint8)[to, r % b.page, h] = b.k.view(torch.uint8)[pg, j % b.page, h]
                vp.view(torch.uint8)[to, r % b.page, h] = b.v.view(torch.uint8)[pg, j % b.page, h]
                w[to, h, r % b.page] = b.weights[pg, h, j % b.page]
    return kept, lens, kp, vp, w


def verify(target, draft, tokens, counts, u_accept, u_sample):
    S, K = tokens.shape
    V = target.shape[2]
    out = torch.full((S, K + 1), -1, dtype=torch.int32)
    accepted = torch.zeros(S, dtype=torch.int32)
    for s in range(S):
        n = min(max(int(counts[s]), 0), K)
        r = 0
        while r < n:
            x = int(tokens[s, r])
            if not 0 <= x < V:
                break
            q = 1.0 if draft is None else draft[s, r, x].double().item()
            if not u_accept[s, r].double().item() * q < target[s, r, x].double().item():
                break
            r += 1
        p = target[s, r].double().clamp(min=0)
        mass = p
        if r < n:
            mass = target[s, r].double().clone()
            if draft is None:
                if 0 <= int(tokens[s, r]) < V:
                    mass[int(tokens[s, r])] = 0
            else:
                mass = mass - draft[s, r].double()
            mass = mass.clamp(min=0)
            if not bool((mass > 0).any()):
                mass = p
        c = torch.cumsum(mass, 0)
        over = torch.nonzero((c > u_sample[s].double() * c[-1]) & (mass > 0))
        has = torch.nonzero(mass > 0)
        pick = over[0, 0] if len(over) else (has[-1, 0] if len(has) else V - 1)
        out[s, :r] = tokens[s, :r]
        out[s, r] = int(pick)
        accepted[s] = r
    return out, accepted
