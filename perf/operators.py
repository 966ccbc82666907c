"""Cases that measure the paged key/value cache: appending to it, attention over it, eviction from it, and the
verification of drafted tokens.

A case's ``kind`` names the operator.  ``run`` computes it in plain torch operations where ``own`` is false, and
through the package's entry points where it is true; ``exact`` computes it from the definition in 64 bits.

Conventions (those of the entry points): sequence s holds ``lens[s]`` slots, its ``starts[s+1] - starts[s]`` new tokens
last; slot j lies in row ``j % page`` of page ``page_table[s, j // page]``; table entries past the length are -1.
"""
import math
import random

import torch

own = False

TYPES = {"bfloat16": torch.bfloat16, "float16": torch.float16, "float8_e4m3fn": torch.float8_e4m3fn}


def listed():
    return [
        # one generated token in each of 64 running conversations
        dict(name="append_step", kind="append", seqs=64, new=1, length=250, ragged=True, heads=8, dim=128, page=16,
             dtype="bfloat16", cache="bfloat16", weights=False),
        # a long prompt taken in at once, with the weights of its slots cleared
        dict(name="append_prompt", kind="append", seqs=1, new=16384, length=20000, ragged=False, heads=8, dim=128, page=64,
             dtype="bfloat16", cache="bfloat16", weights=True),
        # the next token of one short conversation: latency
        dict(name="attend_one_short", kind="attend", seqs=1, new=1, length=1000, ragged=False, heads=32, kv_heads=8, dim=128,
             page=16, dtype="bfloat16", cache="bfloat16", window=0, weights=False),
        # the next token after a very long document: one sequence has to fill the card
        dict(name="attend_one_long", kind="attend", seqs=1, new=1, length=131071, ragged=False, heads=32, kv_heads=8, dim=128,
             page=64, dtype="bfloat16", cache="bfloat16", window=0, weights=False),
        # four drafted tokens in each of 64 conversations, over an 8-bit cache
        dict(name="attend_draft_e4m3", kind="attend", seqs=64, new=4, length=8192, ragged=True, heads=32, kv_heads=8, dim=128,
             page=32, dtype="bfloat16", cache="float8_e4m3fn", window=0, weights=False),
        # a step of 32 conversations that keeps the attention weights for a later eviction
        dict(name="attend_step_weights", kind="attend", seqs=32, new=1, length=8000, ragged=True, heads=32, kv_heads=8, dim=128,
             page=16, dtype="bfloat16", cache="bfloat16", window=0, weights=True),
        # a chunk of a long prompt after its earlier chunks
        dict(name="attend_chunk", kind="attend", seqs=1, new=4096, length=16384, ragged=False, heads=32, kv_heads=8, dim=128,
             page=64, dtype="bfloat16", cache="bfloat16", window=0, weights=False),
        # prompts of several users together: odd lengths, odd pages, small heads, a window, weights kept
        dict(name="attend_window_weights", kind="attend", seqs=9, new=777, length=5001, ragged=True, heads=16, kv_heads=4, dim=64,
             page=24, dtype="float16", cache="float16", window=1024, weights=True),
        # one slot over budget after a generated token
        dict(name="evict_step", kind="evict", seqs=4, length=1025, ragged=False, heads=8, dim=128, page=16, dtype="bfloat16",
             budget=1024, sink=4, recent=64),
        # prompts of eight users cut to an eighth of the slots
        dict(name="evict_prompts", kind="evict", seqs=8, length=32768, ragged=True, heads=8, dim=128, page=64, dtype="bfloat16",
             budget=4096, sink=4, recent=512),
        # four drafted tokens of one conversation
        dict(name="verify_one", kind="verify", seqs=1, drafts=4, vocab=32000, ragged=False, given=True),
        # seven drafted tokens in each of 64 conversations, large vocabulary
        dict(name="verify_batch", kind="verify", seqs=64, drafts=7, vocab=131072, ragged=True, given=True),
    ]


def _log(rng, low, high):
    """A whole number between low and high, spread over its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.4)))))))


def _fits(case, most):
    w = work(case)
    if case["kind"] == "attend":
        # the plain form holds every score of the padded batch
        if case["seqs"] * case["heads"] * case["new"] * case["length"] > 32 * 4096 * 16384:
            return False
        if case["seqs"] * case["kv_heads"] * case["length"] * case["dim"] > 64 * 8 * 8192 * 128:
            return False
    return w["bytes"] <= most["bytes"] and w["flops"] <= most["flops"]


def draw(rng):
    kind = rng.choice(["attend", "attend", "attend", "append", "evict", "verify"])
    dtype = rng.choice(["bfloat16", "bfloat16", "float16"])
    page = rng.choice([16, 16, 20, 24, 32, 64, 128])
    dim = rng.choice([64, 96, 128, 128, 256])
    ragged = rng.random() < 0.6
    if kind == "attend":
        kv = rng.choice([1, 2, 4, 8])
        new = rng.choice([1, 1, rng.randint(2, 9), _log(rng, 10, 4096)])
        case = dict(kind=kind, seqs=_log(rng, 1, 64), new=new, length=max(new, _log(rng, 100, 131071)), ragged=ragged,
                    heads=kv * rng.choice([1, 2, 4, 5, 7, 8]), kv_heads=kv, dim=dim, page=page, dtype=dtype,
                    cache=rng.choice([dtype, dtype, "float8_e4m3fn"]), window=rng.choice([0, 0, 0, _log(rng, 100, 4096)]),
                    weights=rng.random() < 0.4)
    elif kind == "append":
        new = rng.choice([1, rng.randint(2, 9), _log(rng, 10, 16384)])
        case = dict(kind=kind, seqs=_log(rng, 1, 64), new=new, length=new + rng.randint(0, 4000), ragged=ragged,
                    heads=rng.choice([1, 2, 4, 8]), dim=dim, page=page, dtype=dtype, cache=rng.choice([dtype, dtype, "float8_e4m3fn"]),
                    weights=rng.random() < 0.5)
    elif kind == "evict":
        length = _log(rng, 300, 32768)
        budget = _log(rng, 100, length)
        case = dict(kind=kind, seqs=_log(rng, 1, 32), length=length, ragged=ragged, heads=rng.choice([1, 2, 4, 8]), dim=dim,
                    page=page, dtype=dtype, budget=budget, sink=rng.choice([0, 1, 4]), recent=rng.randint(0, budget // 2))
    else:
        return dict(kind=kind, seqs=_log(rng, 1, 64), drafts=rng.randint(1, 7), vocab=_log(rng, 1000, 131072), ragged=ragged,
                    given=rng.random() < 0.75)
    same = [work(c) for c in listed() if c["kind"] == kind]
    most = {k: max(w[k] for w in same) for k in ("bytes", "flops")}
    while not _fits(case, most):
        if case["seqs"] > 1:
            case["seqs"] = (case["seqs"] + 1) // 2
        elif case.get("new", 0) > 1:
            case["new"] = (case["new"] + 1) // 2
        else:
            case["length"] = (case["length"] + 1) // 2
            case["budget"] = min(case.get("budget", 0), case["length"])
    return case if kind == "evict" else {k: v for k, v in case.items() if k != "budget"}


def _lengths(case):
    """(lens, new) of every sequence, from the case alone."""
    rng = random.Random(case["seqs"] * 1000003 + case["length"])
    most = case.get("new", 0)
    lens, new = [], []
    for s in range(case["seqs"]):
        n, m = case["length"], most
        if case["ragged"] and s:
            n = rng.randint(max(1, n // 4), n)
            m = min(n, rng.randint(1, m)) if m else 0
        lens.append(n)
        new.append(m)
    return lens, new


def work(case):
    kind = case["kind"]
    if kind == "verify":
        # one row of the target's and one of the draft's probabilities for every sequence
        return {"bytes": float(case["seqs"] * case["vocab"] * (8 if case["given"] else 4)), "flops": float(3 * case["seqs"] * case["vocab"])}
    lens, new = _lengths(case)
    width = 1 if case.get("cache") == "float8_e4m3fn" else 2
    if kind == "append":
        rows = sum(new) * case["heads"]
        return {"bytes": float(rows * case["dim"] * 2 * (2 + width) + (4 * rows if case["weights"] else 0)), "flops": 0.0}
    if kind == "evict":
        kept = sum(min(n, case["budget"]) for n in lens) * case["heads"]
        return {"bytes": float(4 * sum(lens) * case["heads"] + kept * (2 * case["dim"] * 2 * width + 8)), "flops": 0.0}
    pairs = slots = 0
    for n, m in zip(lens, new):
        w = case["window"] or n
        # query at slot p sees min(p + 1, w) slots
        first, last = n - m, n - 1
        low = min(max(w - 1, first), last + 1)  # slots first .. low-1 see p + 1, the rest w
        pairs += (low - first) * (low + first + 1) // 2 + (last + 1 - low) * w
        slots += min(n, m + w - 1)
    rows = sum(new) * case["heads"]
    data = slots * case["kv_heads"] * 2 * case["dim"] * width + rows * (4 * case["dim"] + 4)
    if case["weights"]:
        data += 4 * sum(lens) * case["kv_heads"]
    return {"bytes": float(data), "flops": float(4 * case["dim"] * case["heads"] * pairs)}


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    kind = case["kind"]
    if kind == "verify":
        S, K, V = case["seqs"], case["drafts"], case["vocab"]
        rng = random.Random(S * 1000003 + V)
        counts = [rng.randint(0, K) if case["ragged"] and s else K for s in range(S)]
        base = normal(S, K + 1, V) * 2.5
        target = torch.softmax(base, -1)
        # a smaller model's distributions, near the target's
        draft = torch.softmax(base[:, :K] + 0.4 * normal(S, K, V), -1)
        tokens = torch.multinomial(draft.reshape(S * K, V), 1, generator=gen).reshape(S, K).to(torch.int32)
        return dict(kind=kind, target=target, draft=draft if case["given"] else None, tokens=tokens,
                    counts=torch.tensor(counts, dtype=torch.int32, device=dev),
                    u_accept=torch.rand((S, K), generator=gen, device=dev), u_sample=torch.rand((S,), generator=gen, device=dev))

    S, ps, D = case["seqs"], case["page"], case["dim"]
    H = case.get("kv_heads", case["heads"])
    lens, new = _lengths(case)
    used = [-(-n // ps) for n in lens]
    more = [-(-min(n, case["budget"]) // ps) for n in lens] if kind == "evict" else [0] * S
    P = sum(used) + sum(more) + 3
    order = torch.randperm(P, generator=gen, device=dev).to(torch.int32)

    def table(first, count):
        rows = max(count)
        at = torch.arange(rows, device=dev)
        n = torch.tensor(count, device=dev)
        base = first + torch.cumsum(n, 0) - n
        return torch.where(at < n[:, None], order[(base[:, None] + at).clamp(max=P - 1)], torch.tensor(-1, dtype=torch.int32, device=dev))

    state = dict(kind=kind, page_table=table(0, used), lens=torch.tensor(lens, dtype=torch.int32, device=dev))
    dtype, cache = TYPES[case["dtype"]], TYPES[case.get("cache", case["dtype"])]
    state["k_scale"] = state["v_scale"] = None
    if cache.itemsize == 1:
        state["k_scale"] = 0.01 + 0.01 * torch.rand((H,), generator=gen, device=dev)
        state["v_scale"] = 0.01 + 0.01 * torch.rand((H,), generator=gen, device=dev)

    def pages(scale):
        x = normal(P, ps, H, D)
        if scale is not None:
            x = (x / scale[:, None]).clamp(-448, 448)
        return x.to(cache)

    state["k_pages"], state["v_pages"] = pages(state["k_scale"]), pages(state["v_scale"])
    state["weights"] = None
    if kind == "evict" or case["weights"]:
        # accumulated weights: few slots hold most of them, and some hold exactly none
        w = torch.rand((P, H, ps), generator=gen, device=dev)
        state["weights"] = torch.where(w < 0.05, torch.zeros_like(w), w.log().square())
    if kind == "evict":
        state.update(new_table=table(sum(used), more), budget=case["budget"], sink=min(case["sink"], case["budget"]),
                     recent=min(case["recent"], case["budget"] - min(case["sink"], case["budget"])))
        return state
    starts = [0]
    for m in new:
        starts.append(starts[-1] + m)
    T = starts[-1]
    state["starts"] = torch.tensor(starts, dtype=torch.int32, device=dev)
    if kind == "append":
        # keys and values come out of one product: rows of a wider matrix
        both = normal(T, 2 * H * D).to(dtype)
        state["k"], state["v"] = both[:, :H * D].view(T, H, D), both[:, H * D:].view(T, H, D)
        return state
    # scores with a standard deviation of 2: neither uniform nor a single slot
    state["q"] = (normal(T, case["heads"], D) * 2).to(dtype)
    state.update(max_q=max(new), max_len=max(lens), window=case["window"], scale=1 / math.sqrt(D))
    return state


def run(state):
    return (_own if own else _plain)[state["kind"]](state)


# ---- the framework's entry points


def _gm():
    import geometric_map_reduce_amd as gm
    return gm


def _own_append(t):
    _gm().keops_cache_append(t["k"], t["v"], t["k_pages"], t["v_pages"], t["page_table"], t["lens"], t["starts"],
                             weights=t["weights"], k_scale=t["k_scale"], v_scale=t["v_scale"])
    return _pages(t)


def _own_attend(t):
    out, lse = _gm().keops_paged_attention(t["q"], t["k_pages"], t["v_pages"], t["page_table"], t["lens"], t["starts"],
                                           t["max_q"], t["max_len"], scale=t["scale"], window=t["window"],
                                           weights=t["weights"], k_scale=t["k_scale"], v_scale=t["v_scale"])
    return dict(out=out, lse=lse, weights=t["weights"])


def _own_evict(t):
    kept, lens = _gm().keops_cache_evict(t["k_pages"], t["v_pages"], t["weights"], t["page_table"], t["lens"],
                                         t["new_table"], t["budget"], sink=t["sink"], recent=t["recent"])
    return dict(kept=kept, lens=lens, **_pages(t))


def _own_verify(t):
    tokens, accepted = _gm().keops_verify_draft(t["target"], t["draft"], t["tokens"], t["counts"], t["u_accept"], t["u_sample"])
    return dict(tokens=tokens, accepted=accepted)


def _pages(t):
    """The cache; what is held in 8 bits as the values it stands for (all of them are 16-bit values too)."""
    k, v = t["k_pages"], t["v_pages"]
    if k.dtype.itemsize == 1:
        k, v = k.to(torch.bfloat16), v.to(torch.bfloat16)
    return dict(k_pages=k, v_pages=v, weights=t["weights"])


_own = dict(append=_own_append, attend=_own_attend, evict=_own_evict, verify=_own_verify)


# ---- plain forms


def _bits(x):
    return x.view(torch.uint8) if x.dtype.itemsize == 1 else x


def _slots(table, ps, count):
    """(page, row) of slots 0 .. count-1 of every sequence."""
    j = torch.arange(count, device=table.device)
    return table[:, j // ps].long().clamp(min=0), (j % ps).expand(table.shape[0], count)


def _owner(starts, T):
    """(sequence, place among its new tokens) of every token."""
    t = torch.arange(T, device=starts.device)
    s = torch.searchsorted(starts[1:].long(), t, right=True)
    return s, t - starts[s]


def _plain_append(t):
    T, ps = t["k"].shape[0], t["k_pages"].shape[1]
    s, i = _owner(t["starts"], T)
    j = (t["lens"][s] - (t["starts"][s + 1] - t["starts"][s]) + i).long()
    page, row = t["page_table"][s, j // ps].long(), j % ps

    def put(pages, x, scale):
        if scale is not None:
            x = (x.float() / scale[:, None]).clamp(-448, 448)
        _bits(pages)[page, row] = _bits(x.to(pages.dtype))

    put(t["k_pages"], t["k"], t["k_scale"])
    put(t["v_pages"], t["v"], t["v_scale"])
    if t["weights"] is not None:
        t["weights"][page, :, row] = 0.0
    return _pages(t)


def _plain_attend(t):
    q, lens, starts, mq, mn = t["q"], t["lens"].long(), t["starts"].long(), t["max_q"], t["max_len"]
    T, Hq, D = q.shape
    S, ps, H = lens.shape[0], t["k_pages"].shape[1], t["k_pages"].shape[2]
    G = Hq // H
    page, row = _slots(t["page_table"], ps, mn)
    k, v = t["k_pages"][page, row].float(), t["v_pages"][page, row].float()  # [S, mn, H, D]
    if t["k_scale"] is not None:
        k, v = k * t["k_scale"][:, None], v * t["v_scale"][:, None]
    i = torch.arange(mq, device=q.device)
    n_new = starts[1:] - starts[:-1]
    qp = q[(starts[:-1, None] + i).clamp(max=T - 1)].float()  # [S, mq, Hq, D]
    qp = qp.reshape(S, mq, H, G, D).permute(0, 2, 3, 1, 4).reshape(S, H, G * mq, D)
    score = torch.matmul(qp, k.permute(0, 2, 3, 1).contiguous()).mul_(t["scale"]).view(S, H, G, mq, mn)
    at = (lens - n_new)[:, None] + i  # slot of every query
    j = torch.arange(mn, device=q.device)
    seen = (j <= at[..., None]) & (i < n_new[:, None])[..., None]
    if t["window"]:
        seen &= j > at[..., None] - t["window"]
    score = score.masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    lse = (total.log() + top).squeeze(-1)  # [S, H, G, mq]
    p = p.div_(torch.where(total > 0, total, torch.ones_like(total)))
    out = torch.matmul(p.view(S, H, G * mq, mn), v.permute(0, 2, 1, 3).contiguous()).view(S, H, G, mq, D)
    s, i = _owner(t["starts"], T)
    out = out.permute(0, 3, 1, 2, 4)[s, i].reshape(T, Hq, D).to(q.dtype)
    lse = lse.permute(0, 3, 1, 2)[s, i].reshape(T, Hq)
    if t["weights"] is not None:
        w = p.sum((2, 3)).permute(0, 2, 1)  # [S, mn, H]
        # slots past a sequence's length go back where they came from
        old = t["weights"][page, :, row]
        last = torch.zeros_like(page)
        real = j < lens[:, None]
        w0 = torch.where(real[..., None], w, torch.zeros_like(w))
        page, row = torch.where(real, page, page[:, :1]), torch.where(real, row, last)
        w0 = torch.where(real[..., None], w0, w0[:, :1])
        t["weights"][page, :, row] = w0.to(old.dtype)
    return dict(out=out, lse=lse, weights=t["weights"])


def _plain_evict(t):
    lens, budget, sink, recent = t["lens"].long(), t["budget"], t["sink"], t["recent"]
    S, ps = lens.shape[0], t["k_pages"].shape[1]
    page, row = _slots(t["page_table"], ps, t["page_table"].shape[1] * ps)
    w = t["weights"][page, :, row].permute(0, 2, 1)  # [S, H, n]
    j = torch.arange(w.shape[-1], device=w.device)
    n = lens[:, None, None]
    w = torch.where((j < sink) | (j >= n - recent), torch.full_like(w, math.inf), w)
    w = torch.where(j < n, w, torch.full_like(w, -math.inf))
    H, most = w.shape[1], w.shape[-1]
    best = torch.sort(w, dim=-1, descending=True, stable=True).indices[..., :budget]
    best = torch.where(torch.arange(best.shape[-1], device=w.device) < n, best, torch.full_like(best, most))
    kept = torch.sort(best, dim=-1).values
    if kept.shape[-1] < budget:
        kept = torch.cat([kept, kept.new_full((S, H, budget - kept.shape[-1]), most)], -1)
    there = kept < most
    new_lens = torch.minimum(lens, torch.full_like(lens, budget))
    src = torch.where(there, kept, kept[..., :1])  # past the end: row 0 again, to slot 0 again
    r = torch.arange(budget, device=w.device)
    dst = torch.where(there, r, torch.zeros_like(r))
    s = torch.arange(S, device=w.device)[:, None, None]
    h = torch.arange(H, device=w.device)[:, None]
    sp, dp = t["page_table"][s, src // ps].long(), t["new_table"][s, dst // ps].long()
    for name in ("k_pages", "v_pages"):
        _bits(t[name])[dp, dst % ps, h] = _bits(t[name])[sp, src % ps, h]
    t["weights"][dp, h, dst % ps] = t["weights"][sp, h, src % ps]
    kept = torch.where(there, kept, torch.full_like(kept, -1))
    return dict(kept=kept.to(torch.int32), lens=new_lens.to(torch.int32), **_pages(t))


def _plain_verify(t):
    p, q, x, n = t["target"], t["draft"], t["tokens"].long(), t["counts"].long()
    S, K = x.shape
    px = p[:, :K].gather(-1, x[..., None]).squeeze(-1).double()
    qx = torch.ones_like(px) if q is None else q.gather(-1, x[..., None]).squeeze(-1).double()
    i = torch.arange(K, device=p.device)
    ok = (t["u_accept"].double() * qx < px) & (i < n[:, None])
    taken = torch.cumprod(ok.long(), -1).sum(-1)  # [S]
    s = torch.arange(S, device=p.device)
    last = p[s, taken].double()
    at = taken.clamp(max=K - 1)
    other = torch.zeros_like(last).scatter_(-1, x[s, at][:, None], 1.0) if q is None else q[s, at].double()
    rest = (last - other).clamp(min=0)
    whole = (taken >= n) | (rest.sum(-1) == 0)
    rest = torch.where(whole[:, None], last.clamp(min=0), rest)
    run_sum = rest.cumsum(-1)
    goal = t["u_sample"].double() * run_sum[:, -1]
    pick = (run_sum <= goal[:, None]).sum(-1).clamp(max=p.shape[-1] - 1)
    i = torch.arange(K + 1, device=p.device)
    xs = torch.cat([x, x[:, :1]], -1)
    tokens = torch.where(i < taken[:, None], xs, torch.where(i == taken[:, None], pick[:, None], torch.full_like(xs, -1)))
    return dict(tokens=tokens.to(torch.int32), accepted=taken.to(torch.int32))


_plain = dict(append=_plain_append, attend=_plain_attend, evict=_plain_evict, verify=_plain_verify)


# ---- from the definitions, in 64 bits


def exact(case, seed):
    t = prepare(case, seed)
    if case["kind"] == "attend":
        return _exact_attend(t)
    if case["kind"] == "evict":
        return _exact_evict(t)
    if case["kind"] == "append":
        return _exact_append(t)
    return _exact_verify(t)


def _rows_of(t, name, s, h, n, table="page_table"):
    """Slots 0 .. n-1 of sequence s and head h in 64 bits, [n, D]."""
    ps = t[name].shape[1]
    ids = t[table][s, :-(-n // ps)].long()
    x = t[name][ids][:, :, h].to(torch.float64).reshape(-1, t[name].shape[-1])[:n]
    scale = t["k_scale" if name == "k_pages" else "v_scale"]
    return x if scale is None else x * scale[h].double()


def _exact_attend(t):
    q, ps = t["q"], t["k_pages"].shape[1]
    T, Hq, D = q.shape
    H = t["k_pages"].shape[2]
    G = Hq // H
    out = torch.zeros((T, Hq, D), dtype=torch.float64, device=q.device)
    lse = torch.zeros((T, Hq), dtype=torch.float64, device=q.device)
    weights = None if t["weights"] is None else t["weights"].double()
    lens, starts = t["lens"].tolist(), t["starts"].tolist()
    for s, n in enumerate(lens):
        a, b = starts[s], starts[s + 1]
        ids = t["page_table"][s, :-(-n // ps)].long()
        for h in range(H):
            k, v = _rows_of(t, "k_pages", s, h, n), _rows_of(t, "v_pages", s, h, n)
            mass = torch.zeros(n, dtype=torch.float64, device=q.device)
            for c in range(a, b, 1024):
                e = min(b, c + 1024)
                x = q[c:e, h * G:(h + 1) * G].double().reshape(-1, D)
                z = (x @ k.T) * t["scale"]
                p = torch.arange(n - b + c, n - b + e, device=q.device).repeat_interleave(G)[:, None]
                j = torch.arange(n, device=q.device)[None]
                hidden = j > p
                if t["window"]:
                    hidden |= p - j >= t["window"]
                z[hidden] = -math.inf
                z_lse = torch.logsumexp(z, 1)
                prob = torch.exp(z - z_lse[:, None])
                out[c:e, h * G:(h + 1) * G] = (prob @ v).reshape(e - c, G, D)
                lse[c:e, h * G:(h + 1) * G] = z_lse.reshape(e - c, G)
                mass += prob.sum(0)
            if weights is not None:
                flat = torch.arange(n, device=q.device)
                weights[ids[flat // ps], h, flat % ps] = mass
    return dict(out=out, lse=lse, weights=weights)


def _exact_append(t):
    ps, lens, starts = t["k_pages"].shape[1], t["lens"].tolist(), t["starts"].tolist()
    held = t["k_scale"] is not None
    got = {}
    for name in ("k", "v"):
        pages = t[name + "_pages"].to(torch.float64)
        x = t[name].double()
        if held:
            # the 8-bit value nearest to the quotient, which the inputs' 32-bit quotient decides
            x = (t[name].float() / t[name + "_scale"][:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).to(torch.float64)
        for s, n in enumerate(lens):
            m = starts[s + 1] - starts[s]
            j = torch.arange(n - m, n, device=x.device)
            pages[t["page_table"][s].long()[j // ps], j % ps] = x[starts[s]:starts[s + 1]]
        got[name + "_pages"] = pages
    weights = None
    if t["weights"] is not None:
        weights = t["weights"].double()
        for s, n in enumerate(lens):
            j = torch.arange(n - (starts[s + 1] - starts[s]), n, device=weights.device)
            weights[t["page_table"][s].long()[j // ps], :, j % ps] = 0
    return dict(got, weights=weights)


def _exact_evict(t):
    ps, lens = t["k_pages"].shape[1], t["lens"].tolist()
    k_pages, v_pages, weights = t["k_pages"].double(), t["v_pages"].double(), t["weights"].double()
    budget, sink, recent = t["budget"], t["sink"], t["recent"]
    for s, n in enumerate(lens):
        j = torch.arange(n, device=weights.device)
        old = t["page_table"][s].long()[j // ps]
        for h in range(weights.shape[1]):
            keep = j
            if n > budget:
                w = weights[old, h, j % ps][sink:n - recent]
                rank = torch.argsort(-w, stable=True)[:budget - sink - recent] + sink
                keep = torch.cat([j[:sink], rank.sort().values, j[n - recent:]])
            r = torch.arange(len(keep), device=weights.device)
            to, at = t["new_table"][s].long()[r // ps], old[keep]
            k_pages[to, r % ps, h] = t["k_pages"][at, keep % ps, h].double()
            v_pages[to, r % ps, h] = t["v_pages"][at, keep % ps, h].double()
            weights[to, h, r % ps] = t["weights"][at, h, keep % ps].double()
    return dict(kept=None, lens=None, k_pages=k_pages, v_pages=v_pages, weights=weights)


def _exact_verify(t):
    S, K = t["tokens"].shape
    tokens = torch.full((S, K + 1), -1, dtype=torch.int32, device=t["target"].device)
    accepted = torch.zeros(S, dtype=torch.int32, device=t["target"].device)
    drafts, counts = t["tokens"].tolist(), t["counts"].tolist()
    for s in range(S):
        r = 0
        while r < counts[s]:
            x = drafts[s][r]
            q = 1.0 if t["draft"] is None else float(t["draft"][s, r, x])
            if not float(t["u_accept"][s, r]) * q < float(t["target"][s, r, x]):
                break
            r += 1
        p = t["target"][s, r].double()
        if r < counts[s]:
            left = p.clone()
            if t["draft"] is None:
                left[drafts[s][r]] = 0
            else:
                left -= t["draft"][s, r].double()
            left[left < 0] = 0
            p = left if bool((left > 0).any()) else p
        c = torch.cumsum(p, 0)
        pick = torch.searchsorted(c, t["u_sample"][s].double() * c[-1], right=True).clamp(max=len(c) - 1)
        tokens[s, :r] = t["tokens"][s, :r]
        tokens[s, r] = pick
        accepted[s] = r
    return dict(tokens=tokens, accepted=accepted)
