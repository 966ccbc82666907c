"""Cases that measure the parts of a serving step around the paged key/value cache: rotary positions, the append that
rotates on the way into a 16-bit, 8-bit or 4-bit cache, attention over a cache held in 4 bits, and the adjustment of
logits by penalties, biases and masks.

A case's ``kind`` names the operator.  ``run`` computes it in plain torch operations where ``own`` is false, and
through the package's entry points where it is true; ``exact`` computes it from the definition in 64 bits.

Conventions (those of the entry points): sequence s holds ``lens[s]`` slots (or tokens of text), its
``starts[s+1] - starts[s]`` new ones last; slot j lies in row ``j % page`` of page ``page_table[s, j // page]``.

A 4-bit cache: blocks of 32 columns share a power of two (a byte b stands for 2^(b - 127), 255 for NaN), an element is
one of 0, 0.5, 1, 1.5, 2, 3, 4, 6 with a sign, two to a byte, the first in the low half.  Pages hold the bytes
[pages, page, heads, dim / 2], scales the powers [pages, heads, page, dim / 32].
"""
import math
import random

import torch

own = False

TYPES = {"bfloat16": torch.bfloat16, "float16": torch.float16, "float32": torch.float32, "float8_e4m3fn": torch.float8_e4m3fn,
         "float4_e2m1": torch.float4_e2m1fn_x2}
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # queries and keys of a decoding step of 16 conversations, rotated where they lie in the wide product's rows
        dict(name="rotary_step", kind="rotary", tokens=16, heads=40, dim=128, rot=128, dtype="bfloat16", interleaved=False,
             scaled=False, inverse=False),
        # a training step's gradient with respect to queries and keys of four texts of 4,096 tokens: the inverse rotation
        dict(name="rotary_gradient", kind="rotary", tokens=16384, heads=40, dim=128, rot=128, dtype="bfloat16", interleaved=True,
             scaled=True, inverse=True),
        # one generated token in each of 64 conversations, rotated on its way into a 16-bit cache
        dict(name="append_step", kind="append", seqs=64, new=1, length=250, ragged=True, heads=32, kv_heads=8, dim=128, rot=128,
             page=16, dtype="bfloat16", cache="bfloat16", interleaved=False, scaled=False, given=False, weights=False),
        # a long prompt into a 4-bit cache, far into a text (positions given), half of each head rotated
        dict(name="append_prompt_4bit", kind="append", seqs=1, new=16384, length=16384, ragged=False, heads=32, kv_heads=8, dim=128,
             rot=64, page=64, dtype="bfloat16", cache="float4_e2m1", interleaved=True, scaled=True, given=True, weights=True),
        # prompts of several users together into a 4-bit cache: odd lengths, odd pages
        dict(name="append_users_4bit", kind="append", seqs=9, new=777, length=900, ragged=True, heads=16, kv_heads=4, dim=96,
             rot=96, page=24, dtype="float16", cache="float4_e2m1", interleaved=False, scaled=False, given=False, weights=False),
        # the next token of one short conversation over a 4-bit cache: latency
        dict(name="attend_one_short", kind="attend", seqs=1, new=1, length=1000, ragged=False, heads=32, kv_heads=8, dim=128, page=16,
             dtype="bfloat16", window=0, weights=False),
        # the next token after a very long document: one sequence has to fill the card
        dict(name="attend_one_long", kind="attend", seqs=1, new=1, length=131071, ragged=False, heads=32, kv_heads=8, dim=128,
             page=64, dtype="bfloat16", window=0, weights=False),
        # four drafted tokens in each of 64 conversations
        dict(name="attend_draft", kind="attend", seqs=64, new=4, length=8192, ragged=True, heads=32, kv_heads=8, dim=128, page=32,
             dtype="bfloat16", window=0, weights=False),
        # a chunk of a long prompt after its earlier chunks
        dict(name="attend_chunk", kind="attend", seqs=1, new=4096, length=16384, ragged=False, heads=32, kv_heads=8, dim=128, page=64,
             dtype="bfloat16", window=0, weights=False),
        # prompts of several users: odd lengths, odd pages, small heads, a window, the slots' weights kept
        dict(name="attend_window_weights", kind="attend", seqs=9, new=777, length=5001, ragged=True, heads=16, kv_heads=4, dim=64,
             page=24, dtype="float16", window=1024, weights=True),
        # one conversation's next token: all penalties, a few biases, a grammar
        dict(name="logits_one", kind="logits", seqs=1, new=1, vocab=32000, length=1000, ragged=False, dtype="float32", penalties=True,
             biases=16, mask=True),
        # four drafted tokens in each of 64 conversations over a large vocabulary
        dict(name="logits_batch", kind="logits", seqs=64, new=4, vocab=131072, length=4096, ragged=True, dtype="bfloat16",
             penalties=True, biases=64, mask=True),
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
    if case["kind"] == "logits" and case["seqs"] * case["new"] * case["length"] > 64 * 4 * 8192:
        return False
    return w["bytes"] <= most["bytes"] and w["flops"] <= most["flops"]


def draw(rng):
    kind = rng.choice(["attend", "attend", "attend", "append", "append", "rotary", "logits"])
    dtype = rng.choice(["bfloat16", "bfloat16", "float16"])
    page = rng.choice([16, 16, 20, 24, 32, 64, 128])
    dim = rng.choice([64, 96, 128, 128, 256])
    ragged = rng.random() < 0.6
    if kind == "attend":
        kv = rng.choice([1, 2, 4, 8])
        new = rng.choice([1, 1, rng.randint(2, 9), _log(rng, 10, 4096)])
        case = dict(kind=kind, seqs=_log(rng, 1, 64), new=new, length=max(new, _log(rng, 100, 131071)), ragged=ragged,
                    heads=kv * rng.choice([1, 2, 4, 5, 7, 8]), kv_heads=kv, dim=dim, page=page, dtype=dtype,
                    window=rng.choice([0, 0, 0, _log(rng, 100, 4096)]), weights=rng.random() < 0.4)
    elif kind == "append":
        kv = rng.choice([1, 2, 4, 8])
        new = rng.choice([1, rng.randint(2, 9), _log(rng, 10, 16384)])
        case = dict(kind=kind, seqs=_log(rng, 1, 64), new=new, length=new + rng.randint(0, 1000), ragged=ragged,
                    heads=kv * rng.choice([1, 2, 4, 5]), kv_heads=kv, dim=dim, rot=rng.choice([dim, dim // 2, 2 * rng.randint(1, dim // 2)]),
                    page=page, dtype=dtype, cache=rng.choice([dtype, "float8_e4m3fn", "float4_e2m1", "float4_e2m1"]),
                    interleaved=rng.random() < 0.5, scaled=rng.random() < 0.5, given=rng.random() < 0.5, weights=rng.random() < 0.5)
    elif kind == "rotary":
        dim = rng.choice([dim, 8 * rng.randint(1, 40), 2 * rng.randint(1, 100)])
        case = dict(kind=kind, tokens=_log(rng, 1, 16384), heads=rng.randint(1, 40), dim=dim,
                    rot=rng.choice([dim, dim // 4 * 2 or 2, 2 * rng.randint(1, dim // 2)]), dtype=rng.choice([dtype, "float32"]),
                    interleaved=rng.random() < 0.5, scaled=rng.random() < 0.5, inverse=rng.random() < 0.5)
    else:
        case = dict(kind=kind, seqs=_log(rng, 1, 64), new=rng.choice([1, 1, rng.randint(2, 8)]), vocab=_log(rng, 1000, 131072),
                    length=_log(rng, 10, 32768), ragged=ragged, dtype=rng.choice([dtype, "float32"]), penalties=rng.random() < 0.8,
                    biases=rng.choice([0, rng.randint(1, 300)]), mask=rng.random() < 0.7)
    same = [work(c) for c in listed() if c["kind"] == kind]
    most = {k: max(w[k] for w in same) for k in ("bytes", "flops")}
    while not _fits(case, most):
        if case.get("seqs", 1) > 1:
            case["seqs"] = (case["seqs"] + 1) // 2
        elif kind == "rotary":
            case["tokens"] = (case["tokens"] + 1) // 2
        elif case["new"] > 1:
            case["new"] = (case["new"] + 1) // 2
        else:
            case["length"] = (case["length"] + 1) // 2
    if kind in ("append", "attend", "logits"):
        case["length"] = max(case["length"], case["new"])
    return case


def _lengths(case):
    """(lens, new) of every sequence, from the case alone."""
    rng = random.Random(case["seqs"] * 1000003 + case["length"])
    lens, new = [], []
    for s in range(case["seqs"]):
        n, m = case["length"], min(case["new"], case["length"])
        if case["ragged"] and s:
            n = rng.randint(max(1, n // 4), n)
            m = min(n, rng.randint(1, m))
        lens.append(n)
        new.append(m)
    return lens, new


def _width(name):
    """Bytes of an element, the shared powers of 4-bit blocks among them."""
    return {"float4_e2m1": 0.5 + 1 / 32, "float8_e4m3fn": 1, "float32": 4}.get(name, 2)


def work(case):
    kind, width = case["kind"], _width(case["dtype"])
    if kind == "rotary":
        n = case["tokens"] * case["heads"]
        # a rotated column takes two products and a sum
        return {"bytes": float(2 * n * case["dim"] * width + 4 * case["tokens"]), "flops": float(3 * n * case["rot"])}
    lens, new = _lengths(case)
    T = sum(new)
    if kind == "logits":
        data = 2 * T * case["vocab"] * width + (T * case["vocab"] / 8 if case["mask"] else 0)
        data += 4 * sum(lens) * case["penalties"] + 8 * case["seqs"] * case["biases"]
        return {"bytes": float(data), "flops": float(2 * T * case["vocab"])}
    held = _width(case.get("cache", "float4_e2m1"))
    if kind == "append":
        rows, slots = T * case["kv_heads"] * case["dim"], _pool(case) * case["page"] * case["kv_heads"] * case["dim"]
        data = T * case["heads"] * case["dim"] * 4 + rows * 2 * (2 + held) + (4 * T * case["kv_heads"] if case["weights"] else 0)
        if held != 2:
            # what is held in 4 or 8 bits is read back as the values it stands for
            data += 2 * slots * (held + 2)
        return {"bytes": float(data), "flops": float(3 * T * (case["heads"] + case["kv_heads"]) * case["rot"])}
    pairs = slots = 0
    for n, m in zip(lens, new):
        w = case["window"] or n
        # query at slot p sees min(p + 1, w) slots
        first, last = n - m, n - 1
        low = min(max(w - 1, first), last + 1)  # slots first .. low-1 see p + 1, the rest w
        pairs += (low - first) * (low + first + 1) // 2 + (last + 1 - low) * w
        slots += min(n, m + w - 1)
    rows = T * case["heads"]
    data = slots * case["kv_heads"] * 2 * case["dim"] * held + rows * (4 * case["dim"] + 4)
    if case["weights"]:
        data += 4 * sum(lens) * case["kv_heads"]
    return {"bytes": float(data), "flops": float(4 * case["dim"] * case["heads"] * pairs)}


def _pool(case):
    """Pages of the pool: those of all sequences and three more."""
    return sum(-(-n // case["page"]) for n in _lengths(case)[0]) + 3


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    kind, dtype = case["kind"], TYPES[case["dtype"]]
    state = dict(kind=kind)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device=dev)

    if kind in ("rotary", "append"):
        n = case["rot"] // 2
        freqs = 500000.0 ** (-torch.arange(n, dtype=torch.float64, device=dev) / n)
        if case["scaled"]:
            # a text eight times as long: slow pairs turn an eighth as fast, the fastest as before
            keep = (torch.log2(freqs * 8192 / (2 * math.pi)) / 5).clamp(0, 1)
            freqs = freqs * (keep + (1 - keep) / 8)
        state.update(freqs=freqs, factor=1.2 if case["scaled"] else 1.0, interleaved=case["interleaved"])
    if kind == "rotary":
        T, H, D = case["tokens"], case["heads"], case["dim"]
        # queries and keys beside the values, as they come out of one product
        state["x"] = normal(T, H + 3, D).to(dtype)[:, :H]
        state["positions"] = torch.arange(T, dtype=torch.int32, device=dev) % 4096 + int(torch.randint(0, 4096, (1,), generator=gen, device=dev))
        state["inverse"] = case["inverse"]
        return state

    S = case["seqs"]
    lens, new = _lengths(case)
    T = sum(new)
    starts = [0]
    for m in new:
        starts.append(starts[-1] + m)
    state.update(lens=torch.tensor(lens, dtype=torch.int32, device=dev), starts=torch.tensor(starts, dtype=torch.int32, device=dev))
    if kind == "logits":
        V, W = case["vocab"], max(lens)
        state["logits"] = (normal(T, V) * 3).to(dtype)
        state.update({k: None for k in ("tokens", "prompt_lens", "repetition", "presence", "frequency", "bias_tokens", "bias", "mask")})
        if case["penalties"]:
            # a text repeats its common words
            state["tokens"] = (V * uniform(S, W) ** 4).to(torch.int32).clamp(max=V - 1)
            state["prompt_lens"] = torch.tensor([n // 3 for n in lens], dtype=torch.int32, device=dev)
            state["repetition"], state["presence"], state["frequency"] = 1 + 0.3 * uniform(S), uniform(S), 0.5 * uniform(S)
        if case["biases"]:
            B = case["biases"]
            at = (uniform(S, 1) * V).long() + torch.arange(B, device=dev) * max(1, V // B)
            state["bias_tokens"] = torch.where(uniform(S, B) < 0.1, torch.full_like(at, -1), at % V).to(torch.int32)
            state["bias"] = normal(S, B) * 4
        if case["mask"]:
            words = torch.randint(-2 ** 31, 2 ** 31, (T, -(-V // 32)), generator=gen, device=dev).to(torch.int32)
            words[uniform(T) < 0.05] = 0  # a grammar that is at its end
            state["mask"] = words
        return state

    ps, D, H = case["page"], case["dim"], case["kv_heads"]
    cache = TYPES[case.get("cache", "float4_e2m1")]
    used = [-(-n // ps) for n in lens]
    P = _pool(case)
    order = torch.randperm(P, generator=gen, device=dev).to(torch.int32)
    at, count = torch.arange(max(used), device=dev), torch.tensor(used, device=dev)
    base = torch.cumsum(count, 0) - count
    state["page_table"] = torch.where(at < count[:, None], order[(base[:, None] + at).clamp(max=P - 1)],
                                      torch.tensor(-1, dtype=torch.int32, device=dev))
    for name in ("k", "v"):
        x, scale = normal(P, ps, H, D), None
        if cache == torch.float4_e2m1fn_x2:
            codes, power = _to_4bit(x, _top(dtype))
            x, scale = codes.view(cache), power.permute(0, 2, 1, 3).contiguous().view(torch.float8_e8m0fnu)
        elif cache.itemsize == 1:
            scale = 0.01 + 0.01 * uniform(H)
            x = (x / scale[:, None]).clamp(-448, 448).to(cache)
        state[name + "_pages"], state[name + "_scale"] = x.to(cache), scale
    state["weights"] = None
    if case["weights"]:
        # accumulated weights: few slots hold most of them, and some hold exactly none
        w = uniform(P, H, ps)
        state["weights"] = torch.where(w < 0.05, torch.zeros_like(w), w.log().square())
    if kind == "append":
        wide = normal(T, case["heads"] + 2 * H, D).to(dtype)
        state.update(q=wide[:, :case["heads"]], k=wide[:, case["heads"]:-H], v=wide[:, -H:], positions=None)
        if case["given"]:
            far = int(torch.randint(0, 1 << 18, (1,), generator=gen, device=dev))
            state["positions"] = torch.arange(T, dtype=torch.int32, device=dev) + far
        # the whole pool as one sequence
        state.update(all_pages=torch.arange(P, dtype=torch.int32, device=dev)[None], slots=P * ps,
                     all_lens=torch.tensor([P * ps], dtype=torch.int32, device=dev),
                     all_starts=torch.tensor([0, P * ps], dtype=torch.int32, device=dev))
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


def _own_rotary(t):
    return _gm().keops_rotary(t["x"], t["positions"], t["freqs"], interleaved=t["interleaved"], factor=t["factor"], inverse=t["inverse"])


def _own_append(t):
    gm = _gm()
    q = gm.keops_cache_append_rotary(t["q"], t["k"], t["v"], t["k_pages"], t["v_pages"], t["page_table"], t["lens"], t["starts"],
                                     t["freqs"], positions=t["positions"], interleaved=t["interleaved"], factor=t["factor"],
                                     weights=t["weights"], k_scale=t["k_scale"], v_scale=t["v_scale"])
    k, v = t["k_pages"], t["v_pages"]
    if t["k_scale"] is not None:
        k, v = gm.keops_cache_read(k, v, t["all_pages"], t["all_lens"], t["all_starts"], t["slots"], dtype=t["q"].dtype,
                                   k_scale=t["k_scale"], v_scale=t["v_scale"])
    return dict(q=q, k=k, v=v, weights=t["weights"])


def _own_attend(t):
    out, lse = _gm().keops_paged_attention(t["q"], t["k_pages"], t["v_pages"], t["page_table"], t["lens"], t["starts"], t["max_q"],
                                           t["max_len"], scale=t["scale"], window=t["window"], weights=t["weights"],
                                           k_scale=t["k_scale"], v_scale=t["v_scale"])
    return dict(out=out, lse=lse, weights=t["weights"])


def _own_logits(t):
    return _gm().keops_adjust_logits(t["logits"], t["starts"], tokens=t["tokens"], lens=t["lens"], prompt_lens=t["prompt_lens"],
                                     repetition=t["repetition"], presence=t["presence"], frequency=t["frequency"],
                                     bias_tokens=t["bias_tokens"], bias=t["bias"], mask=t["mask"])


_own = dict(rotary=_own_rotary, append=_own_append, attend=_own_attend, logits=_own_logits)


# ---- plain forms


def _top(dtype):
    """The largest power of a 4-bit block: no element is past the 16-bit type's largest number."""
    return 140 if dtype == torch.float16 else 252


def _to_4bit(x, top):
    """(bytes, powers) of the 4-bit blocks of x, in 64 bits: the least power under which nothing rounds past 6."""
    x = x.reshape(*x.shape[:-1], -1, 32).double()
    most = x.abs().amax(-1)
    part, e = torch.frexp(most)
    b = torch.where(most > 0, e.long() - 1 + (part >= 0.875).long() - 2 + 127, torch.zeros_like(e, dtype=torch.long)).clamp(0, top)
    lost = ~torch.isfinite(x).all(-1)
    y = x * ((1023 + 127 - b) << 52).view(torch.float64)[..., None]
    y = torch.where(lost[..., None], torch.zeros_like(y), y)
    a = y.abs()
    # halfway goes to the even code
    code = ((a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte() + (a > 2.5).byte() + (a >= 3.5).byte() +
            (a > 5).byte()) | (torch.signbit(y).byte() << 3)
    code = code.flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), torch.where(lost, torch.full_like(b, 255), b).to(torch.uint8)


def _from_4bit(codes, powers):
    """The values of 4-bit bytes [.., dim / 2] under powers [.., dim / 32]."""
    level = torch.tensor(LEVELS + tuple(-x for x in LEVELS), device=codes.device)
    both = torch.stack([level.repeat(16), level.repeat_interleave(16)], -1)  # of a byte
    x = both[codes.int()].flatten(-2)
    two = torch.where(powers == 255, torch.full_like(powers, 0, dtype=torch.float32) + math.nan, (powers.int() << 23).view(torch.float32))
    return (x.unflatten(-1, (-1, 32)) * two[..., None]).flatten(-2)


def _to_8bit(x):
    """x (64 bits, finite) to the nearest e4m3 value, in 32 bits: steps of an eighth of the power of two, of 2^-9 below 2^-6."""
    e = torch.frexp(x).exponent.long().clamp(min=-5) - 4
    step = ((1023 + e) << 52).view(torch.float64)
    return (torch.round(x / step) * step).float()


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


def _rotated(x, positions, t, wide, inverse=False):
    """x [tokens, heads, dim] rotated; angles in 64 bits, the rest in 64 (wide) or 32."""
    n = t["freqs"].shape[0]
    angle = positions.double()[:, None] * t["freqs"]
    c, s = torch.cos(angle) * t["factor"], torch.sin(angle) * (-t["factor"] if inverse else t["factor"])
    x = x.double() if wide else x.float()
    c, s = c.to(x.dtype)[:, None], s.to(x.dtype)[:, None]
    a, b = (x[..., 0:2 * n:2], x[..., 1:2 * n:2]) if t["interleaved"] else (x[..., :n], x[..., n:2 * n])
    a, b = a * c - b * s, a * s + b * c
    turned = torch.stack([a, b], -1).flatten(-2) if t["interleaved"] else torch.cat([a, b], -1)
    return torch.cat([turned, x[..., 2 * n:]], -1)


def _plain_rotary(t):
    return _rotated(t["x"], t["positions"], t, False, t["inverse"]).to(t["x"].dtype)


def _plain_append(t):
    T, ps = t["k"].shape[0], t["k_pages"].shape[1]
    s, i = _owner(t["starts"], T)
    j = (t["lens"][s] - (t["starts"][s + 1] - t["starts"][s]) + i).long()
    page, row = t["page_table"][s, j // ps].long(), j % ps
    at = j if t["positions"] is None else t["positions"]
    dtype, scale = t["q"].dtype, t["k_scale"]
    # borders between 4-bit and 8-bit values are met in 64 bits
    k = _rotated(t["k"], at, t, scale is not None)
    got = {}
    for name, x in (("k", k), ("v", t["v"])):
        pages, scale = t[name + "_pages"], t[name + "_scale"]
        if pages.dtype == torch.float4_e2m1fn_x2:
            codes, power = _to_4bit(x, _top(dtype))
            _bits(pages)[page, row] = codes
            _bits(scale)[page, :, row] = power
            got[name] = _from_4bit(_bits(pages), _bits(scale).permute(0, 2, 1, 3)).to(dtype).flatten(0, 1)
        elif scale is not None:
            x = (_to_8bit(x / scale[:, None].double()) if name == "k" else x.float() / scale[:, None]).clamp(-448, 448)
            _bits(pages)[page, row] = _bits(x.to(pages.dtype))
            got[name] = (pages.float() * scale[:, None]).to(dtype).flatten(0, 1)
        else:
            pages[page, row] = x.to(pages.dtype)
            got[name] = pages
    if t["weights"] is not None:
        t["weights"][page, :, row] = 0.0
    return dict(q=_rotated(t["q"], at, t, False).to(dtype), **got, weights=t["weights"])


def _plain_attend(t):
    q, lens, starts, mq, mn = t["q"], t["lens"].long(), t["starts"].long(), t["max_q"], t["max_len"]
    T, Hq, D = q.shape
    S, ps, H = lens.shape[0], t["k_pages"].shape[1], t["k_pages"].shape[2]
    G = Hq // H
    page, row = _slots(t["page_table"], ps, mn)
    k, v = (_from_4bit(_bits(t[x + "_pages"])[page, row], _bits(t[x + "_scale"])[page, :, row]) for x in "kv")  # [S, mn, H, D]
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
        # places past a sequence's length write its first slot again
        real = j < lens[:, None]
        w = torch.where(real[..., None], w, w[:, :1])
        page, row = torch.where(real, page, page[:, :1]), torch.where(real, row, torch.zeros_like(row))
        t["weights"][page, :, row] = w
    return dict(out=out, lse=lse, weights=t["weights"])


def _plain_logits(t):
    z, starts = t["logits"].float(), t["starts"]
    T, V = z.shape
    s, i = _owner(starts, T)
    j = (t["lens"][s] - (starts[s + 1] - starts[s]) + i).long()
    if t["tokens"] is not None:
        text = t["tokens"][s].long()
        at = torch.arange(text.shape[1], device=z.device)
        there = (at <= j[:, None]) & (text >= 0) & (text < V)
        made = there & (at >= t["prompt_lens"][s, None])
        text = text.clamp(0, V - 1)
        seen = torch.zeros((T, V), dtype=torch.int32, device=z.device).scatter_add_(1, text, there.int())
        times = torch.zeros((T, V), dtype=torch.int32, device=z.device).scatter_add_(1, text, made.int()).float()
        r = t["repetition"][s, None]
        z = torch.where(seen > 0, torch.where(z > 0, z / r, z * r), z)
        z = z - t["frequency"][s, None] * times - torch.where(times > 0, t["presence"][s, None], torch.zeros_like(r))
    if t["bias"] is not None:
        ids = t["bias_tokens"][s].long()
        there = (ids >= 0) & (ids < V)
        # the ids of a list differ; what is no id goes to a column of its own
        add = torch.zeros((T, V + 1), device=z.device).scatter_(1, torch.where(there, ids, torch.full_like(ids, V)), t["bias"][s])
        z = z + add[:, :V]
    if t["mask"] is not None:
        x = torch.arange(V, device=z.device)
        allowed = (t["mask"][:, x // 32] >> (x % 32).int()) & 1
        z = z.masked_fill(allowed == 0, -math.inf)
    return z.to(t["logits"].dtype)


_plain = dict(rotary=_plain_rotary, append=_plain_append, attend=_plain_attend, logits=_plain_logits)


# ---- from the definitions, in 64 bits


def exact(case, seed):
    t = prepare(case, seed)
    return dict(rotary=_exact_rotary, append=_exact_append, attend=_exact_attend, logits=_exact_logits)[case["kind"]](t)


def _turn(x, positions, t, sign=1.0):
    """As a product of complex numbers."""
    n = t["freqs"].shape[0]
    x = x.double()
    angle = sign * positions.double()[:, None, None] * t["freqs"]
    by = torch.polar(torch.full_like(angle, t["factor"]), angle)
    x = x.clone()
    if t["interleaved"]:
        z = torch.complex(x[..., 0:2 * n:2], x[..., 1:2 * n:2]) * by
        x[..., 0:2 * n:2], x[..., 1:2 * n:2] = z.real, z.imag
    else:
        z = torch.complex(x[..., :n], x[..., n:2 * n]) * by
        x[..., :n], x[..., n:2 * n] = z.real, z.imag
    return x


def _exact_rotary(t):
    return _turn(t["x"], t["positions"], t, -1.0 if t["inverse"] else 1.0)


def _nearest_4bit(x, top):
    """The values that blocks of 32 columns of x (64 bits, finite) are held as."""
    level = torch.tensor(LEVELS, dtype=torch.float64, device=x.device)
    b = x.unflatten(-1, (-1, 32))
    most = b.abs().amax(-1, keepdim=True)
    power = torch.full_like(most, float(top - 127))
    e = torch.floor(torch.log2(most.clamp(min=2.0 ** -200)))
    e = torch.where(most < torch.exp2(e), e - 1, e)
    e = torch.where(most >= torch.exp2(e + 1), e + 1, e)
    e = e - 2
    e = torch.where(most >= 7 * torch.exp2(e), e + 1, e).clamp(min=-127)
    power = torch.where(most > 0, torch.minimum(power, e), torch.full_like(e, -127.0))
    y = b / torch.exp2(power)
    away = (y.abs()[..., None] - level).abs()
    # of two that are equally near the one with the even code
    odd = torch.arange(8, device=x.device) % 2
    near = (away.amin(-1, keepdim=True) == away) & ~((odd == 1) & ((away == away.amin(-1, keepdim=True)).sum(-1, keepdim=True) > 1))
    value = (near * level).amax(-1)
    return (torch.copysign(value, y) * torch.exp2(power)).flatten(-2)


def _nearest_8bit(x):
    """The e4m3 values nearest to x (64 bits, finite), cut to +-448."""
    level = torch.arange(127, dtype=torch.uint8, device=x.device).view(torch.float8_e4m3fn).double()
    middle = (level[1:] + level[:-1]) / 2
    low, high = (torch.bucketize(x.abs(), middle, right=r) for r in (False, True))  # they differ halfway
    return torch.copysign(level[torch.where(low % 2 == 0, low, high)], x)


def _held(t, name):
    """The pool's values in 64 bits, [pages, page, heads, dim]."""
    pages, scale = t[name + "_pages"], t[name + "_scale"]
    if pages.dtype != torch.float4_e2m1fn_x2:
        return pages.double() if scale is None else pages.double() * scale.double()[:, None]
    raw, level = pages.view(torch.uint8), torch.tensor(LEVELS, dtype=torch.float64, device=pages.device)
    code = torch.stack([raw & 15, raw >> 4], -1).flatten(-2).long()
    value = level[code % 8] * torch.where(code < 8, 1.0, -1.0)
    power = torch.exp2(scale.view(torch.uint8).double() - 127).permute(0, 2, 1, 3)
    return value * power.repeat_interleave(32, -1)


def _exact_append(t):
    ps, lens, starts = t["k_pages"].shape[1], t["lens"].tolist(), t["starts"].tolist()
    T, cache = t["k"].shape[0], t["k_pages"].dtype
    at = t["positions"]
    if at is None:
        at = torch.cat([torch.arange(n - (b - a), n, device=t["k"].device) for n, a, b in zip(lens, starts, starts[1:])])
    k, v = _turn(t["k"], at, t), t["v"].double()
    weights = None if t["weights"] is None else t["weights"].double()
    got = {}
    for name, x in (("k", k), ("v", v)):
        pages, scale = _held(t, name), t[name + "_scale"]
        if cache == torch.float4_e2m1fn_x2:
            x = torch.cat([_nearest_4bit(x[c:c + 1024], _top(t["q"].dtype)) for c in range(0, T, 1024)])
        elif scale is not None:
            x = _nearest_8bit(x / scale.double()[:, None]) * scale.double()[:, None]
        for s, n in enumerate(lens):
            j = torch.arange(n - (starts[s + 1] - starts[s]), n, device=x.device)
            page = t["page_table"][s].long()[j // ps]
            pages[page, j % ps] = x[starts[s]:starts[s + 1]]
            if weights is not None:
                weights[page, :, j % ps] = 0
        got[name] = pages if scale is None else pages.flatten(0, 1)
    return dict(q=_turn(t["q"], at, t), **got, weights=weights)


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
        part = {x + y: _bits(t[x + y])[ids].view(t[x + y].dtype) for x in "kv" for y in ("_pages", "_scale")}
        ks, vs = (_held(part, x).flatten(0, 1)[:n] for x in "kv")
        for h in range(H):
            k, v = ks[:, h], vs[:, h]
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


def _exact_logits(t):
    z = t["logits"].double()
    V = z.shape[1]
    lens, starts = t["lens"].tolist(), t["starts"].tolist()
    for s, n in enumerate(lens):
        for r in range(starts[s], starts[s + 1]):
            j = n - starts[s + 1] + r
            if t["tokens"] is not None:
                text = t["tokens"][s, :j + 1].long()
                made = torch.bincount(text[int(t["prompt_lens"][s]):], minlength=V)[:V]
                x = torch.unique(text)
                old = z[r, x]
                rep = t["repetition"][s].double()
                z[r, x] = torch.where(old > 0, old / rep, old * rep)
                z[r] -= t["frequency"][s].double() * made + t["presence"][s].double() * (made > 0)
            if t["bias"] is not None:
                ids = t["bias_tokens"][s].long()
                z[r, ids[ids >= 0]] += t["bias"][s][ids >= 0].double()
            if t["mask"] is not None:
                bit = (t["mask"][r].long()[:, None] >> torch.arange(32, device=z.device)) & 1
                z[r, bit.flatten()[:V] == 0] = -math.inf
    return z
