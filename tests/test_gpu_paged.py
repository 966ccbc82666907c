"""The paged key/value cache and draft verification on the GPU, through the binding, against plain
64-bit forms (paged_reference.py).  Tolerances are the bounds derived there: half a step of the
16-bit type for the output and for each p, fp32 sums, and what the exponential makes of them."""
from __future__ import annotations

import sys

import pytest
import torch

import paged_reference as ref

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import geometric_map_reduce_amd as gm

BF, FP, E4 = torch.bfloat16, torch.float16, torch.float8_e4m3fn


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def say(msg):
    print(msg, flush=True)
    sys.stdout.flush()


def put(t):
    return None if t is None else t.cuda()


def run_attention(b, decay=0.0, **kw):
    w = put(b.weights)
    out, lse = gm.keops_paged_attention(put(b.q), put(b.k), put(b.v), put(b.table), put(b.lens_t()), put(b.starts),
                                        max(b.new + [0]), max(b.lens + [0]), scale=b.scale, window=b.window, weights=w,
                                        decay=decay, k_scale=put(b.k_scale), v_scale=put(b.v_scale), **kw)
    torch.cuda.synchronize()
    return out.cpu(), lse.cpu(), None if w is None else w.cpu()


def close(got, want, tol, what):
    got, want = got.double(), want.double()
    same = (got == want) | (got.isnan() & want.isnan())
    bad = ~(same | ((got - want).abs() <= tol))
    if bool(bad.any()):
        i = tuple(torch.nonzero(bad)[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: {got[i].item()} for "
                             f"{want[i].item()}, tolerance {tol[i].item() if torch.is_tensor(tol) else tol}")


def check_attention(b, decay=0.0, **kw):
    out, lse, w = run_attention(b, decay, **kw)
    o, z, ww, ot, zt, wt = ref.attention(b, decay)
    close(lse, z, zt, "lse")
    close(out, o, ot, "out")
    if w is not None:
        close(w, ww, wt, "weights")


# lens, new tokens, query heads, key/value heads, dim, page, type, cache, window
CASES = [
    ([1], [1], 1, 1, 64, 16, BF, BF, 0),
    ([1], [1], 8, 2, 128, 16, FP, E4, 0),
    ([33], [1], 4, 1, 128, 16, BF, BF, 0),
    ([1000], [1], 32, 8, 128, 16, BF, BF, 0),
    ([1000, 1, 77, 513], [1, 1, 1, 1], 8, 2, 64, 20, FP, FP, 0),
    ([300, 129, 4000], [4, 2, 3], 8, 2, 128, 32, BF, E4, 0),
    ([300, 0, 40], [4, 0, 3], 10, 2, 96, 24, FP, E4, 0),       # a sequence without slots
    ([700, 64], [9, 1], 14, 2, 96, 7, BF, BF, 0),              # pages that end inside a tile; 63 rows
    ([500, 31], [3, 2], 7, 1, 256, 64, BF, BF, 100),
    ([260], [1], 5, 1, 256, 128, FP, E4, 33),
    ([200, 90], [4, 3], 8, 1, 256, 16, FP, FP, 0),             # 32 rows
    ([64, 65, 63], [64, 65, 63], 4, 2, 64, 16, BF, BF, 0),     # whole prompts
    ([130, 257], [130, 200], 4, 1, 128, 24, FP, FP, 0),
    ([300], [150], 2, 1, 96, 128, BF, E4, 0),
    ([333, 80], [40, 80], 8, 2, 256, 20, BF, BF, 0),
    ([222], [60], 8, 1, 256, 16, FP, E4, 17),
    ([2000], [12], 8, 1, 128, 64, BF, BF, 0),                  # many-rows form, split over the slots
    ([777, 400, 100], [300, 10, 100], 8, 4, 64, 24, FP, FP, 128),
    ([1500], [5], 8, 8, 128, 1, BF, BF, 64),                   # one slot a page
]


@pytest.mark.parametrize("lens,new,heads,kv,dim,page,dtype,cache,window", CASES)
@pytest.mark.parametrize("weights", [False, True])
def test_attention(lens, new, heads, kv, dim, page, dtype, cache, window, weights):
    say(f"attention {lens} {new} {heads}/{kv} {dim} page {page} {dtype} {cache} window {window} weights {weights}")
    b = ref.Batch(hash((len(lens), sum(lens), dim)) & 0xffff, lens, new, heads, kv, dim, page, dtype, cache)
    b.window = window
    if weights:
        b.weights = torch.full((b.P, kv, page), float("nan"))
    check_attention(b)


@pytest.mark.parametrize("new", [1, 50])
def test_weights_accumulate(new):
    say(f"weights accumulate, {new} new tokens")
    b = ref.Batch(5, [150, 90], [new, new], 8, 2, 128, 16)
    b.weights = torch.rand((b.P, 2, 16), generator=b.gen)
    check_attention(b, decay=1.0)
    check_attention(b, decay=0.5)


@pytest.mark.parametrize("dim,new,cache", [(64, 3, BF), (128, 3, E4), (96, 3, BF), (256, 3, BF), (64, 40, BF), (128, 40, E4),
                                           (256, 40, BF), (96, 40, FP)])
def test_hidden_values_reach_no_row(dim, new, cache):
    """NaN and infinities in the key and value of a later token, and below the window, change nothing
    for the rows that do not see them; the rows that see them get what the formula gives."""
    say(f"hidden non-finite values, dim {dim}, {new} new, {cache}")
    dtype = FP if cache == FP else BF
    b = ref.Batch(9, [140], [new], 4, 2, dim, 16, dtype, cache)
    b.window = 101
    nan = torch.tensor(float("nan")).to(cache)

    def spot(j):
        return b.table[0, j // 16].item(), j % 16
    for j in (140 - 1, 140 - new - 100, 140 - new + 1):       # the last token, below the window, a middle one
        pg, row = spot(j)
        b.v.view(torch.uint8 if cache == E4 else torch.int16)[pg, row, :, 3] = nan.view(torch.uint8 if cache == E4 else torch.int16)
        if cache != E4:
            b.v[pg, row, :, 7] = float("inf")
    pg, row = spot(140 - 1)
    b.k.view(torch.uint8 if cache == E4 else torch.int16)[pg, row, 0, 0] = nan.view(torch.uint8 if cache == E4 else torch.int16)
    out, lse, _ = run_attention(b)
    # reference: token by token, only what it sees
    o, z, _, ot, zt, _ = ref.attention(b)
    first = 140 - new
    for t in range(new):
        sees = [j for j in (139, 140 - new - 100, 140 - new + 1) if j <= first + t and j > first + t - 101]
        for h in range(4):
            if not sees:
                assert bool(out[t, h].isfinite().all()) and bool(lse[t, h].isfinite())
                close(out[t, h], o[t, h], ot[t, h], f"row {t}")
            else:
                assert out[t, h].isnan().equal(o[t, h].isnan()), (t, h)
                fin = o[t, h].isfinite()
                close(out[t, h][fin], o[t, h][fin], ot[t, h][fin], f"row {t}")
                assert (out[t, h] == float("inf")).equal(o[t, h] == float("inf"))


@pytest.mark.parametrize("new", [2, 30])
def test_absent_pages(new):
    """Entries outside the pool are slots that are not there; a row that sees none has 0 and -inf."""
    say(f"absent pages, {new} new")
    b = ref.Batch(11, [100, 64], [new, new], 8, 2, 64, 16)
    b.weights = torch.rand((b.P, 2, 16), generator=b.gen)
    b.table[0, 1] = -1
    b.table[0, 3] = b.P
    b.table[1, :4] = 2 ** 31 - 1
    check_attention(b)
    out, lse, _ = run_attention(b)
    assert bool((out[new:] == 0).all()) and bool((lse[new:] == -float("inf")).all())
    # a table that is too narrow: the rest is absent too
    b.table = b.table[:, :5].contiguous()
    check_attention(b)


def test_fewer_slots_than_new_tokens():
    """A token before the first slot sees nothing."""
    for new in (4, 70):
        say(f"{new} new tokens, 3 slots")
        b = ref.Batch(3, [3], [new], 2, 1, 64, 16)
        check_attention(b)


@pytest.mark.parametrize("new", [1, 33])
def test_strides(new):
    """Keys and values interleaved in one pool, heads outside slots, queries inside wider rows."""
    say(f"strides, {new} new")
    b = ref.Batch(13, [90, 41], [new, min(new, 41)], 8, 2, 128, 16, junk=0.0)
    want = run_attention(b)
    both = torch.stack([b.k, b.v], 1).cuda()                   # [P, 2, ps, H, D]
    heads = torch.stack([b.k, b.v], 1).transpose(2, 3).contiguous().cuda().transpose(2, 3)   # [P, 2, H, ps, D] as above
    wide = torch.randn((b.T, 3, 8, 128)).to(BF)
    wide[:, 1] = b.q
    q = wide.cuda()[:, 1]
    for pool in (both, heads):
        out, lse = gm.keops_paged_attention(q, pool[:, 0], pool[:, 1], put(b.table), put(b.lens_t()), put(b.starts), new, 90)
        torch.cuda.synchronize()
        assert torch.equal(out.cpu(), want[0]) and torch.equal(lse.cpu(), want[1])


def test_far_pages():
    """Byte offsets past 2^32 in the pool."""
    say("far pages")
    b = ref.Batch(17, [70], [2], 8, 4, 128, 16, junk=0.0)
    P = (5 << 30) // (16 * 4 * 128 * 2)
    k = torch.zeros((P, 16, 4, 128), dtype=BF, device="cuda")
    v = torch.zeros_like(k)
    far = torch.arange(P - b.table.shape[1], P, dtype=torch.int32)
    k[far.long().cuda()] = b.k.cuda()[b.table[0].long().cuda()]
    v[far.long().cuda()] = b.v.cuda()[b.table[0].long().cuda()]
    w = torch.zeros((P, 4, 16), device="cuda")
    out, lse = gm.keops_paged_attention(put(b.q), k, v, far[None].cuda(), put(b.lens_t()), put(b.starts), 2, 70, weights=w)
    o, z, _, ot, zt, _ = ref.attention(b)
    close(out.cpu(), o, ot, "out")
    close(lse.cpu(), z, zt, "lse")
    assert abs(w.sum().item() - 2 * 8) < 1e-3
    # the last slots again, with other values
    nk, nv = torch.randn((2, 4, 128)).to(BF), torch.randn((2, 4, 128)).to(BF)
    gm.keops_cache_append(nk.cuda(), nv.cuda(), k, v, far[None].cuda(), put(b.lens_t()), put(b.starts))
    assert torch.equal(k[P - 1, 4:6].cpu(), nk) and torch.equal(v[P - 1, 4:6].cpu(), nv)
    kept, _ = gm.keops_cache_evict(k, v, w, far[None].cuda(), put(b.lens_t()), torch.tensor([[0]], dtype=torch.int32).cuda(), 16,
                                   sink=1, recent=2)
    assert torch.equal(k[0, 14:16].cpu(), nk) and kept[0, 0, 15].item() == 69


def test_other_stream_and_outputs():
    say("another stream, given outputs")
    b = ref.Batch(19, [500, 300], [1, 1], 8, 2, 128, 16)
    want = run_attention(b)
    args = [put(t) for t in (b.q, b.k, b.v, b.table, b.lens_t(), b.starts)]
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    out, lse = torch.empty_like(args[0]), torch.empty((2, 8), device="cuda")
    o, z = gm.keops_paged_attention(*args, 1, 500, out=out, lse=lse, stream=st)
    o2, _ = gm.keops_paged_attention(*args, 1, 500, stream=st)
    st.synchronize()
    assert o is out and z is lse
    assert torch.equal(o.cpu(), want[0]) and torch.equal(z.cpu(), want[1]) and torch.equal(o2.cpu(), want[0])


def test_graph():
    """A decoding step captured once and replayed with other contents: every replay equals the eager call."""
    say("graph of a decoding step")
    b = ref.Batch(23, [900, 300], [1, 1], 8, 2, 128, 16, junk=0.0)
    b.weights = torch.zeros((b.P, 2, 16))
    k, v, table, lens, starts, w = (put(t) for t in (b.k, b.v, b.table, b.lens_t(), b.starts, b.weights))
    q, nk, nv = put(b.q), torch.zeros((2, 2, 128), dtype=BF, device="cuda"), torch.zeros((2, 2, 128), dtype=BF, device="cuda")

    def step():
        gm.keops_cache_append(nk, nv, k, v, table, lens, starts, weights=w)
        return gm.keops_paged_attention(q, k, v, table, lens, starts, 1, 900, weights=w, decay=1.0)
    step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            out, lse = step()
    for rep in range(4):
        g = torch.Generator().manual_seed(rep)
        for t in (q, nk, nv):
            t.copy_(torch.randn(t.shape, generator=g).to(BF))
        w.zero_()
        graph.replay()
        torch.cuda.synchronize()
        o, z, ww = out.clone(), lse.clone(), w.clone()
        w.zero_()
        eo, ez = step()
        torch.cuda.synchronize()
        assert torch.equal(o, eo) and torch.equal(z, ez) and torch.equal(ww, w)


def test_results_repeat():
    """The same call gives the same bits."""
    for new in (1, 40):
        say(f"repeat, {new} new")
        b = ref.Batch(29, [2000, 700], [new, new], 8, 2, 128, 16)
        b.weights = torch.zeros((b.P, 2, 16))
        x, y = run_attention(b), run_attention(b)
        assert all(torch.equal(p, q) for p, q in zip(x, y))


# ---- append

@pytest.mark.parametrize("dtype,cache", [(BF, BF), (FP, FP), (BF, E4), (FP, E4)])
@pytest.mark.parametrize("lens,new,heads,dim,page", [([1], [1], 1, 64, 16), ([40, 0, 300, 7], [3, 0, 300, 1], 2, 96, 20),
                                                     ([129] * 70, [1] * 70, 4, 128, 32), ([50, 2], [5, 4], 3, 256, 1)])
@pytest.mark.parametrize("weights", [False, True])
def test_append(dtype, cache, lens, new, heads, dim, page, weights):
    say(f"append {dtype} {cache} {len(lens)} sequences, {heads} x {dim}, page {page}")
    b = ref.Batch(31, lens, new, heads, heads, dim, page, dtype, cache, junk=0.0)
    if weights:
        b.weights = torch.rand((b.P, heads, page), generator=b.gen) + 1
    b.table[0, 0] = b.P + 5 if len(lens) == 4 else b.table[0, 0]
    both = (torch.randn((b.T, 2 * heads * dim), generator=b.gen) * 2).to(dtype)
    both[0, 0], both[0, 1], both[-1, -1] = float("inf"), float("nan"), -1e4
    k, v = both[:, :heads * dim].view(b.T, heads, dim), both[:, heads * dim:].view(b.T, heads, dim)
    kp, vp, w = put(b.k), put(b.v), put(b.weights)
    dev = both.cuda()
    gm.keops_cache_append(dev[:, :heads * dim].view(b.T, heads, dim), dev[:, heads * dim:].view(b.T, heads, dim), kp, vp,
                          put(b.table), put(b.lens_t()), put(b.starts), weights=w, k_scale=put(b.k_scale), v_scale=put(b.v_scale))
    torch.cuda.synchronize()
    rk, rv, rw = ref.append(b, k, v)
    for got, want in ((kp, rk), (vp, rv)):
        got, want = got.cpu().float(), want.float()
        assert torch.equal(got.isnan(), want.isnan())
        assert torch.equal(got.nan_to_num(0.0, 1e9, -1e9), want.nan_to_num(0.0, 1e9, -1e9))
    if weights:
        assert torch.equal(w.cpu(), rw)


def test_append_every_16_bit_value():
    """Each bf16 and fp16 value to the nearest e4m3 of its quotient."""
    for dtype in (BF, FP):
        say(f"append, every {dtype}")
        x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(dtype).reshape(1024, 1, 64)
        b = ref.Batch(37, [1024], [1024], 1, 1, 64, 64, dtype, E4, junk=0.0)
        for scale in (1.0, 0.0173):
            b.k_scale, b.v_scale = torch.tensor([scale]), torch.tensor([1.0])
            kp, vp = put(b.k), put(b.v)
            gm.keops_cache_append(x.cuda(), x.cuda(), kp, vp, put(b.table), put(b.lens_t()), put(b.starts),
                                  k_scale=put(b.k_scale), v_scale=put(b.v_scale))
            got = kp.cpu()[b.table[0].long()].reshape(-1).float()
            want = (x.reshape(-1).float() / scale).clamp(-448, 448).to(E4).float()
            assert torch.equal(got.isnan(), want.isnan())
            assert torch.equal(got.nan_to_num(0.0), want.nan_to_num(0.0))


# ---- eviction

@pytest.mark.parametrize("lens,heads,dim,page,cache,budget,sink,recent", [
    ([1], 1, 64, 16, BF, 1, 0, 0), ([20, 5, 17], 2, 64, 16, BF, 16, 1, 4), ([100, 33], 2, 96, 24, FP, 32, 4, 28),
    ([1025, 900, 0], 2, 128, 16, BF, 600, 4, 64), ([257], 1, 256, 20, E4, 100, 0, 50), ([300, 10], 3, 128, 7, E4, 11, 0, 0),
    ([5000], 1, 64, 64, BF, 4999, 0, 0),
])
@pytest.mark.parametrize("ties", [False, True])
def test_evict(lens, heads, dim, page, cache, budget, sink, recent, ties):
    say(f"evict {lens} {heads} x {dim} page {page} {cache} budget {budget} sink {sink} recent {recent} ties {ties}")
    more = sum(-(-min(n, budget) // page) for n in lens)
    b = ref.Batch(41, lens, [0] * len(lens), heads, heads, dim, page, FP if cache == FP else BF, cache, junk=0.0, spare=more + 1)
    w = torch.rand((b.P, heads, page), generator=b.gen)
    if ties:
        w = (w * 3).floor() / 2
        w[w == 0.5] = -0.0
        w.view(-1)[::13] = float("nan")
        w.view(-1)[::17] = float("inf")
        w.view(-1)[::19] = -1.0
    b.weights = w
    if ties and len(lens) == 2 and page == 24:
        b.table[0, 2] = -1
    width = max(1, max(-(-min(n, budget) // page) for n in lens))
    new = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(lens):
        u = -(-min(n, budget) // page)
        new[s, :u] = b.free[at:at + u]
        at += u
    kp, vp, wp = put(b.k), put(b.v), put(b.weights)
    kept, nl = gm.keops_cache_evict(kp, vp, wp, put(b.table), put(b.lens_t()), put(new), budget, sink=sink, recent=recent)
    torch.cuda.synchronize()
    rkept, rl, rk, rv, rw = ref.evict(b, new, budget, sink, recent)
    assert torch.equal(nl.cpu(), rl)
    assert torch.equal(kept.cpu(), rkept)
    assert torch.equal(kp.cpu().view(torch.uint8), rk.view(torch.uint8))
    assert torch.equal(vp.cpu().view(torch.uint8), rv.view(torch.uint8))
    assert torch.equal(wp.cpu().view(torch.int32), rw.view(torch.int32))


@pytest.mark.parametrize("n", [32768, 40000, 100001])
def test_evict_long(n):
    """Rows that fit the selection's LDS, and that do not."""
    say(f"evict, {n} slots")
    budget, page = 777, 128
    P = -(-n // page) + -(-budget // page)
    g = torch.Generator().manual_seed(n)
    k = torch.randn((P, page, 1, 64), generator=g).to(BF).cuda()
    w = torch.rand((P, 1, page), generator=g)
    w[w < 0.3] = 0.0
    order = torch.randperm(P, generator=g).to(torch.int32)
    table, new = order[:-(-n // page)][None], order[-(-n // page):][None]
    flat = w[table[0].long(), 0].reshape(-1)[:n]
    mid = torch.sort(flat[4:n - 100], descending=True, stable=True).indices[:budget - 104] + 4
    want = torch.cat([torch.arange(4), mid.sort().values, torch.arange(n - 100, n)])
    v = k.clone()
    kept, nl = gm.keops_cache_evict(k, v, w.cuda(), table.cuda(), torch.tensor([n], dtype=torch.int32).cuda(), new.cuda(), budget,
                                    sink=4, recent=100)
    assert torch.equal(kept.cpu()[0, 0].long(), want) and nl.item() == budget
    src = k.cpu()[table[0].long(), :, 0].reshape(-1, 64)[want]
    assert torch.equal(v.cpu()[new[0].long(), :, 0].reshape(-1, 64)[:budget], src)


# ---- verification

def verify_case(seed, S, K, V, near=0.4):
    g = torch.Generator().manual_seed(seed)
    base = torch.randn((S, K + 1, V), generator=g) * 2.5
    target = torch.softmax(base, -1)
    draft = torch.softmax(base[:, :K] + near * torch.randn((S, K, V), generator=g), -1)
    tokens = torch.multinomial(draft.reshape(-1, V), 1, generator=g).reshape(S, K).to(torch.int32) if K else \
        torch.zeros((S, 0), dtype=torch.int32)
    counts = torch.randint(0, K + 1, (S,), generator=g, dtype=torch.int32)
    return target, draft, tokens, counts, torch.rand((S, K), generator=g), torch.rand((S,), generator=g)


def check_verify(target, draft, tokens, counts, ua, us):
    out, acc = gm.keops_verify_draft(put(target), put(draft), put(tokens), put(counts), put(ua), put(us))
    ro, ra = ref.verify(target, draft, tokens, counts, ua, us)
    assert torch.equal(acc.cpu(), ra) and torch.equal(out.cpu(), ro)


@pytest.mark.parametrize("S,K,V", [(1, 1, 1), (1, 4, 1000), (7, 3, 63), (33, 7, 5003), (3, 100, 70), (2, 2, 131072), (4, 0, 333)])
@pytest.mark.parametrize("given", [False, True])
def test_verify(S, K, V, given):
    say(f"verify {S} x {K} of {V}, draft {given}")
    target, draft, tokens, counts, ua, us = verify_case(S * 100 + V, S, K, V)
    check_verify(target, draft if given else None, tokens, counts, ua, us)
    us[0] = 0.0
    counts[:] = K
    check_verify(target, draft if given else None, tokens, counts, ua, us)


def test_verify_edges():
    say("verify, edges")
    target, draft, tokens, counts, ua, us = verify_case(77, 12, 3, 257)
    counts[:] = 3
    tokens[0, 0] = -1                       # refused
    tokens[1, 1] = 257
    counts[2] = -5                          # cut to 0 and to 3
    counts[3] = 99
    draft[4] = target[4, :3]                # nothing left over: never refused but for u = 1
    ua[4] = 1.0
    draft[5] = 0.0                          # always taken
    target[6] = 0.0                         # no mass at all
    target[7, :, 128:] = 0.0
    us[7] = 1.0                             # past every running sum
    target[8, :, :] = 0.0
    target[8, :, 200] = 1.0
    target[9] *= 3.0                        # scale free
    target[10] = 0.0
    target[10, :, [5, 9]] = 0.25            # ties of the running sum with u
    us[10], ua[10] = 0.5, 1.0
    check_verify(target, draft, tokens, counts, ua, us)
    check_verify(target, None, tokens, counts, ua, us)


# ---- wider ranges

def random_case(seed):
    """A seeded case of the operators' ranges, small enough for the plain form."""
    import random
    rng = random.Random(seed)
    kv = rng.choice([1, 2, 4])
    dtype = rng.choice([BF, BF, FP])
    dim = rng.choice([64, 96, 128, 256])
    group = rng.choice([1, 2, 4, 5, 7, 8])
    S = rng.choice([1, 2, 5, 70])
    top = rng.choice([1, 3, 9, 40])
    if S == 70:
        kv, top = 1, rng.choice([1, 2])
    lens, new = [], []
    for _ in range(S):
        n = rng.choice([0, 1, rng.randint(1, 50), rng.randint(1, 700 if S < 70 else 120)])
        lens.append(n)
        new.append(min(n, rng.randint(0, top)))
    return dict(lens=lens, new=new, heads=kv * group, kv_heads=kv, dim=dim, page=rng.choice([1, 5, 16, 20, 64, 128]), dtype=dtype,
                cache=rng.choice([dtype, dtype, E4])), rng.choice([0, 0, 1, 37, 200]), rng.random() < 0.5


@pytest.mark.parametrize("seed", range(40))
def test_attention_random(seed):
    case, window, weights = random_case(seed)
    say(f"random attention {seed}: {len(case['lens'])} sequences, {case['heads']}/{case['kv_heads']} x {case['dim']} page {case['page']} "
        f"{case['dtype']} {case['cache']} window {window} weights {weights} lens {case['lens'][:6]} new {case['new'][:6]}")
    b = ref.Batch(seed, **case)
    if b.T == 0:
        b = ref.Batch(seed, **dict(case, lens=case["lens"] + [9], new=case["new"] + [2]))
    b.window = window
    if weights:
        b.weights = torch.rand((b.P, b.kv, b.page), generator=b.gen)
    check_attention(b, decay=0.25 if weights and seed % 2 else 0.0)


@pytest.mark.parametrize("S", [64, 65, 200])
def test_many_sequences(S):
    """More sequences than a wave has lanes, some of them empty; the second pass joins parts of most."""
    say(f"{S} sequences")
    lens = [(37 * s) % 300 for s in range(S)]
    lens[S // 2] = 3000
    new = [min(n, 1 + s % 2) for s, n in enumerate(lens)]
    b = ref.Batch(S, lens, new, 4, 1, 64, 16)
    b.weights = torch.full((b.P, 1, 16), float("nan"))
    check_attention(b)


@pytest.mark.parametrize("new,weights", [(2, False), (2, True), (20, False)])
def test_negative_and_zero_scale(new, weights):
    for scale in (-0.11, 0.0):
        say(f"scale {scale}, {new} new")
        b = ref.Batch(43, [200, 90], [new, new], 8, 2, 128, 16)
        b.scale = scale
        if weights:
            b.weights = torch.zeros((b.P, 2, 16))
        check_attention(b)


@pytest.mark.parametrize("new", [1, 40])
def test_lengths_past_the_bounds(new):
    """max_len and max_q cut; what is inside them is right."""
    say(f"cut lengths, {new} new")
    b = ref.Batch(47, [300, 100], [new, new], 4, 2, 64, 16)
    out, lse = gm.keops_paged_attention(put(b.q), put(b.k), put(b.v), put(b.table), put(b.lens_t()), put(b.starts), new, 100)
    torch.cuda.synchronize()
    o, z, _, ot, zt, _ = ref.attention(b)
    close(out[new:].cpu(), o[new:], ot[new:], "out")
    close(lse[new:].cpu(), z[new:], zt[new:], "lse")
    if new > 1:
        full = run_attention(b)[0]
        out, _ = gm.keops_paged_attention(put(b.q), put(b.k), put(b.v), put(b.table), put(b.lens_t()), put(b.starts), new // 2, 300)
        torch.cuda.synchronize()
        half = new // 2
        o, _, _, ot, _, _ = ref.attention(b)
        close(out[:half].cpu(), o[:half], ot[:half], "first half")
        assert full.shape == out.shape


@pytest.mark.parametrize("n,budget", [(30000, 25000), (70000, 60000), (70000, 100)])
def test_evict_ties_at_the_border(n, budget):
    """The border falls among thousands of equal weights: the lower slots stay."""
    say(f"evict ties, {n} slots, budget {budget}")
    page = 64
    used, more = -(-n // page), -(-budget // page)
    g = torch.Generator().manual_seed(n + budget)
    w = torch.rand((used + more, 1, page), generator=g)
    w[w < 0.4 if budget > 1000 else w < 2.0] = 0.0
    order = torch.randperm(used + more, generator=g).to(torch.int32)
    flat = w[order[:used].long(), 0].reshape(-1)[:n]
    mid = torch.sort(flat[3:n - 10], descending=True, stable=True).indices[:budget - 13] + 3
    want = torch.cat([torch.arange(3), mid.sort().values, torch.arange(n - 10, n)])
    k = torch.zeros((used + more, page, 1, 64), dtype=BF, device="cuda")
    kept, _ = gm.keops_cache_evict(k, k.clone(), w.cuda(), order[:used][None].cuda(), torch.tensor([n], dtype=torch.int32).cuda(),
                                   order[used:][None].cuda(), budget, sink=3, recent=10)
    assert torch.equal(kept.cpu()[0, 0].long(), want)


def test_verify_graph():
    say("graph of a verification")
    target, draft, tokens, counts, ua, us = (put(t) for t in verify_case(5, 4, 3, 9000))
    gm.keops_verify_draft(target, draft, tokens, counts, ua, us)
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            out, acc = gm.keops_verify_draft(target, draft, tokens, counts, ua, us)
    for rep in range(4):
        new = verify_case(50 + rep, 4, 3, 9000)
        for t, x in zip((target, draft, tokens, counts, ua, us), new):
            t.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        o, a = gm.keops_verify_draft(target, draft, tokens, counts, ua, us)
        ro, ra = ref.verify(*new)
        torch.cuda.synchronize()
        assert torch.equal(out, o) and torch.equal(acc, a) and torch.equal(o.cpu(), ro) and torch.equal(a.cpu(), ra)


@pytest.mark.parametrize("new", [1, 40])
def test_many_small_weights(new):
    """One slot far above 60,000 others, whose weights fp16 cannot hold one by one, but which add up."""
    say(f"many small weights, {new} new")
    n, D = 60000 + new, 64
    b = ref.Batch(61, [n], [new], 1, 1, D, 128, FP)
    one = torch.zeros(D, dtype=FP)
    one[0] = 1.0
    b.q[:] = one * 8
    b.k[:], b.v[:] = 0.0, 1.0
    b.k[b.table[0, 0].item(), 0, 0] = one * 19.0          # exp(19) = 2^27.4 times the others
    b.v[b.table[0, 0].item(), 0, 0] = 0.0
    out, lse = gm.keops_paged_attention(put(b.q), put(b.k), put(b.v), put(b.table), put(b.lens_t()), put(b.starts), new, n, scale=0.125)
    torch.cuda.synchronize()
    import math
    rest = torch.arange(60000, 60000 + new, dtype=torch.float64)
    total = math.exp(19.0) + rest
    # the others' p is 2^-27.4 of the largest, held to 2^-32: 2^-4.6 of itself at most
    assert bool(((out[:, 0, 0].double().cpu() - rest / total).abs() <= rest / total * 2 ** -4.5 + 2 ** -25).all())
    assert bool(((lse[:, 0].double().cpu() - total.log()).abs() <= 19 * 16 * 2 ** -24 + n * 2 ** -24).all())


def test_failed_workspace_enqueues_nothing():
    say("failing workspace")
    b = ref.Batch(53, [900, 500], [1, 1], 8, 2, 128, 16)
    args = [put(t) for t in (b.q, b.k, b.v, b.table, b.lens_t(), b.starts)]
    out, lse = torch.full_like(args[0], 3.0), torch.full((2, 8), 3.0, device="cuda")
    v = [put(t) for t in verify_case(5, 2, 3, 5000)]
    vo, va = torch.full((2, 4), 7, dtype=torch.int32, device="cuda"), torch.full((2,), 7, dtype=torch.int32, device="cuda")
    gm.keops_set_option(gm.KEOPS_OPT_FAIL_ALLOC, 1)
    try:
        with pytest.raises(gm.KeopsError) as e:
            gm.keops_paged_attention(*args, 1, 900, out=out, lse=lse)
        assert e.value.status == -3
        with pytest.raises(gm.KeopsError) as e:
            gm.keops_verify_draft(*v, out=vo, accepted=va)
        assert e.value.status == -3
    finally:
        gm.keops_set_option(gm.KEOPS_OPT_FAIL_ALLOC, 0)
    torch.cuda.synchronize()
    assert bool((out == 3).all()) and bool((lse == 3).all()) and bool((vo == 7).all()) and bool((va == 7).all())
    # a workspace for each call gives the same bits
    want = gm.keops_paged_attention(*args, 1, 900)
    gm.keops_set_option(gm.KEOPS_OPT_WS_CACHE, 2)
    try:
        got = gm.keops_paged_attention(*args, 1, 900)
        torch.cuda.synchronize()
    finally:
        gm.keops_set_option(gm.KEOPS_OPT_WS_CACHE, 0)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("new", [1, 40])
def test_wide_windows_and_long_lengths(new):
    """Windows beyond every slot change nothing; a length beyond all bounds is cut."""
    say(f"wide windows, {new} new")
    b = ref.Batch(59, [140], [new], 4, 2, 64, 16)
    want = run_attention(b)
    for b.window in (140, 2 ** 30 - 1, 2 ** 31 - 1):
        got = run_attention(b)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    b.window = 0
    lens = torch.tensor([2 ** 31 - 1], dtype=torch.int32, device="cuda")
    out, lse = gm.keops_paged_attention(put(b.q), put(b.k), put(b.v), put(b.table), lens, put(b.starts), new, 140)
    torch.cuda.synchronize()
    # every token sees all 140 slots of the table
    n = 140
    k, v = (b.rows(t, None, 0, 0, n)[0] for t in (b.k, b.v))
    p = torch.softmax(b.q[0, 0].double() @ k.T * b.scale, 0)
    assert (out[0, 0].double().cpu() - p @ v).abs().max() <= 2 ** -7 * v.abs().max()


def test_binding_refusals():
    """What the kernels cannot take is named before any launch."""
    b = ref.Batch(1, [20], [2], 4, 2, 64, 16, junk=0.0)
    q, k, v, table, lens, starts = (put(t) for t in (b.q, b.k, b.v, b.table, b.lens_t(), b.starts))

    def attend(**kw):
        a = dict(q=q, k_pages=k, v_pages=v, page_table=table, lens=lens, starts=starts, max_q=2, max_len=20)
        a.update(kw)
        return gm.keops_paged_attention(**a)
    attend()
    wide = torch.zeros((2, 4, 65), dtype=BF, device="cuda")
    for kw, what in [(dict(q=q.float()), "q"), (dict(q=q.half()), "q"), (dict(q=q[:, :3].contiguous()), "multiple"), (dict(q=wide[:, :, 1:]), "q"),
                     (dict(q=q.transpose(0, 1)), "q"), (dict(v_pages=v[:-1]), "v_pages"), (dict(v_pages=v.half()), "v_pages"),
                     (dict(k_pages=k[..., :32], v_pages=v[..., :32]), "dim"), (dict(k_pages=k.float(), v_pages=v.float()), "k_pages"),
                     (dict(page_table=table.long()), "page_table"), (dict(page_table=table[0]), "page_table"), (dict(lens=lens.long()), "lens"),
                     (dict(lens=lens.cpu()), "lens"), (dict(starts=starts[:-1]), "starts"), (dict(max_q=-1), "max_q"),
                     (dict(weights=torch.zeros((3, 2, 16), device="cuda")), "weights"), (dict(k_scale=torch.ones(2, device="cuda")), "float8"),
                     (dict(k_pages=k.to(E4), v_pages=v.to(E4)), "k_scale"), (dict(out=torch.empty_like(q, dtype=torch.float32)), "out"),
                     (dict(lse=torch.empty((2, 4), device="cuda", dtype=BF)), "lse")]:
        with pytest.raises(ValueError, match=what):
            attend(**kw)
    with pytest.raises(gm.KeopsError):
        attend(scale=float("nan"))
    with pytest.raises(gm.KeopsError):
        attend(out=q)
    with pytest.raises(ValueError, match="k must"):
        gm.keops_cache_append(q, q, k, v, table, lens, starts)
    with pytest.raises(ValueError, match="shape and type of k"):
        gm.keops_cache_append(q[:, :2].contiguous(), q[:1, :2].contiguous(), k, v, table, lens, starts)
    w = torch.zeros((b.P, 2, 16), device="cuda")
    for kw in (dict(budget=0), dict(budget=4, sink=3, recent=2), dict(budget=40)):
        with pytest.raises(ValueError):
            gm.keops_cache_evict(k, v, w, table, lens, table[:, :1].contiguous(), **kw)
    with pytest.raises(ValueError, match="weights"):
        gm.keops_cache_evict(k, v, None, table, lens, table, 4)
    target, draft, tokens, counts, ua, us = (put(t) for t in verify_case(5, 2, 3, 50))
    for i, bad in enumerate((target[:, :3].contiguous(), draft.double(), tokens.long(), counts[:1], ua[:, :2].contiguous(), us.double())):
        a = [target, draft, tokens, counts, ua, us]
        a[i] = bad
        with pytest.raises(ValueError):
            gm.keops_verify_draft(*a)


def test_example_decodes():
    """The example's loop: every round's attention equals the dense formula over the cache as it stands, the weights
    have grown by what the rows gave, and evicted caches go on."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "paged_decode.py")
    spec = importlib.util.spec_from_file_location("paged_decode", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    rounds = [0]

    def watch(st):
        rounds[0] += 1
        if rounds[0] % 5:
            return
        m, p = st["model"], st["pages"]
        for s in range(len(st["lens"])):
            n, a, e = int(st["lens"][s]), int(st["starts"][s]), int(st["starts"][s + 1])
            rows = st["table"][s].long()
            k = p.k[rows].reshape(-1, m.kv, m.dim)[:n].double().cpu()
            v = p.v[rows].reshape(-1, m.kv, m.dim)[:n].double().cpu()
            assert torch.equal(k[n - (e - a):], st["k"][a:e].double().cpu())
            q = st["q"][a:e].double().cpu()
            for h in range(m.heads):
                z = q[:, h] @ k[:, h // (m.heads // m.kv)].T / m.dim ** 0.5
                z.masked_fill_(torch.arange(n) > torch.arange(n - (e - a), n)[:, None], -float("inf"))
                o = torch.softmax(z, -1) @ v[:, h // (m.heads // m.kv)]
                assert (st["out"][a:e, h].double().cpu() - o).abs().max() <= 2 ** -7 * v.abs().max()
    text = ex.decode(rounds=40, watch=watch)
    assert rounds[0] == 40 and all(40 <= len(t) <= 160 for t in text)
    assert ex.decode(rounds=10) == [t[:len(u)] for t, u in zip(text, ex.decode(rounds=10))]


@pytest.mark.parametrize("late", [0, 1, 2, 3])
@pytest.mark.parametrize("dim", [64, 96, 128, 256])
def test_nonfinite_value_reaches_every_row_that_sees_it(dim, late):
    """128 rows of one tile, 32 for each wave; the rows of one wave meet a new largest score in the tile that holds
    an infinity and a NaN, so that it is behind the others there."""
    say(f"non-finite values for every row that sees them, dim {dim}, wave {late} late")
    b = ref.Batch(21, [96], [32], 4, 1, dim, 16)
    b.q.zero_()
    b.q[8 * late:8 * late + 8, :, 0] = 16.0

    def spot(j):
        return b.table[0, j // 16].item(), j % 16
    for j in range(96):
        pg, row = spot(j)
        b.k[pg, row, 0, 0] = 1.0 if j < 64 else 64.0
    for j, col, value in ((65, 3, float("inf")), (66, 7, float("nan"))):
        pg, row = spot(j)
        b.v[pg, row, 0, col] = value
    out, lse, _ = run_attention(b)
    o, z, _, ot, zt, _ = ref.attention(b)
    close(lse, z, zt, "lse")
    for t in range(32):
        # slot 65 is seen from token 1 on, slot 66 from token 2
        assert bool((out[t, :, 3] == float("inf")).all()) == (t >= 1), t
        assert bool(out[t, :, 7].isnan().all()) == (t >= 2), t
    rest = [c for c in range(dim) if c not in (3, 7)]
    close(out[..., rest], o[..., rest], ot[..., rest], "out")


@pytest.mark.parametrize("page", [1, 6, 7, 12, 16])
@pytest.mark.parametrize("n,sink,recent", [(40, 0, 0), (700, 3, 5), (4099, 5, 1), (9000, 1, 77), (33000, 2, 3)])
def test_evict_pages_and_sinks(page, n, sink, recent):
    """Quadruples of slots that end inside a page, a sink or the row; weights that are not 16-byte aligned."""
    say(f"eviction, {n} slots, page {page}, sink {sink}, recent {recent}")
    budget = max(sink + recent + 1, n // 3)
    g = torch.Generator().manual_seed(n + page)
    used, kept_pages = -(-n // page), -(-budget // page)
    P = used + kept_pages
    order = torch.randperm(P, generator=g).to(torch.int32)
    table, new = order[:used][None].clone(), order[used:][None].clone()
    table[0, used // 2] = -1                                         # a page that is not there
    store = torch.zeros(P * page + 1, device="cuda")
    w = store[1:].view(P, 1, page) if page == 16 else torch.zeros((P, 1, page), device="cuda")
    flat = torch.randint(0, max(2, n // 50), (n,), generator=g).float() + 1
    j = torch.arange(n)
    w.copy_(torch.zeros((P, page)).index_put_((order[:used].long()[j // page], j % page), flat).view(P, 1, page))
    k = torch.randn((P, page, 1, 64), generator=g).to(BF).cuda()
    v = k.clone()
    lens = torch.tensor([n], dtype=torch.int32).cuda()
    kept, new_lens = gm.keops_cache_evict(k, v, w, table.cuda(), lens, new.cuda(), budget, sink=sink, recent=recent)
    torch.cuda.synchronize()
    flat[(j // page) == used // 2] = -float("inf")                   # absent: the smallest
    middle = torch.argsort(-flat[sink:n - recent], stable=True)[:budget - sink - recent] + sink
    want = torch.cat([j[:sink], middle.sort().values, j[n - recent:]])
    assert torch.equal(kept[0, 0].cpu().long(), want) and new_lens.item() == budget


@pytest.mark.parametrize("new", [1, 40])
def test_infinite_key_of_weight_zero(new):
    """A key that every row's score sends to -infinity has no part in any output, and a weight of exactly 0."""
    say(f"infinite key, {new} new")
    b = ref.Batch(67, [300], [new], 2, 1, 64, 16)
    b.q[:, :, 0] = -b.q[:, :, 0].abs() - 1
    b.k[b.table[0, 0].item(), 3, 0, 0] = float("inf")
    b.weights = torch.ones((b.P, 1, 16))
    out, lse, w = run_attention(b)
    assert w[b.table[0, 0].item(), 0, 3].item() == 0
    assert bool(out.isfinite().all()) and bool(lse.isfinite().all())
    total = sum(w[b.table[0, j // 16].item(), 0, j % 16].item() for j in range(300))
    assert abs(total - 2 * new) <= 2 * new * 2 ** -16


@pytest.mark.parametrize("dtype", [BF, FP])
def test_append_e4m3_scales(dtype):
    """Every 16-bit value over scales of all kinds equals the value nearest to the fp32 quotient."""
    say(f"e4m3 quotients, {dtype}")
    g = torch.Generator().manual_seed(71)
    bits = (torch.randint(0, 1 << 23, (40,), generator=g) + (torch.randint(100, 150, (40,), generator=g) << 23)).to(torch.int32)
    special = [1.0, -0.5, 3.0, 2.0 ** -61, 2.0 ** -60, 2.0 ** 60, 2.0 ** 61, 1e-38, 1e-42, 3e38, float("inf"), float("nan"), 0.0,
               float(torch.tensor(0x3fffffff, dtype=torch.int32).view(torch.float32)), float(torch.tensor(0x3f7fffff, dtype=torch.int32).view(torch.float32))]
    x = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(dtype).view(-1, 1, 64).cuda()
    T = x.shape[0]
    table, lens = torch.arange(T // 16, dtype=torch.int32, device="cuda")[None], torch.tensor([T], dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    for i, s in enumerate(bits.view(torch.float32).tolist() + special):
        scale = torch.tensor([s], device="cuda")
        k = torch.zeros((T // 16, 16, 1, 64), device="cuda").to(E4)
        v = torch.zeros_like(k)
        gm.keops_cache_append(x, x, k, v, table, lens, starts, k_scale=scale, v_scale=torch.ones_like(scale))
        want = (x.float() / scale).clamp(-448, 448).to(E4).view(torch.uint8).view(-1)
        got = k.view(torch.uint8).view(-1)
        nan = (want & 0x7f) == 0x7f
        assert torch.equal(got[~nan], want[~nan]) and bool(((got[nan] & 0x7f) == 0x7f).all()), (i, s)


@pytest.mark.parametrize("dtype,cache", [(BF, BF), (FP, FP), (BF, E4), (FP, E4)])
@pytest.mark.parametrize("dim", [64, 96, 128, 256])
@pytest.mark.parametrize("new,weights", [(1, False), (2, True), (7, False), (6, True)])
def test_loads_past_the_caches(dtype, cache, dim, new, weights):
    """The bounds of a call, not its lengths, say that its keys and values may be more than a cache holds."""
    say(f"loads past the caches, {dtype} {cache}, dim {dim}, {new} new, weights {weights}")
    lens = [300, 77, 40]
    b = ref.Batch(73, lens, [new, 1, 0], 8, 2, dim, 24, dtype, cache)
    if weights:
        b.weights = torch.zeros((b.P, 2, 24))
    w = put(b.weights)
    most = 1 << 19                                          # 2 x 3 x 2 x 2^19 rows: 402 MB and more
    out, lse = gm.keops_paged_attention(put(b.q), put(b.k), put(b.v), put(b.table), put(b.lens_t()), put(b.starts), new, most,
                                        weights=w, k_scale=put(b.k_scale), v_scale=put(b.v_scale))
    torch.cuda.synchronize()
    o, z, ww, ot, zt, wt = ref.attention(b)
    close(lse.cpu(), z, zt, "lse")
    close(out.cpu(), o, ot, "out")
    if weights:
        close(w.cpu(), ww, wt, "weights")


def test_eviction_past_the_caches():
    say("eviction with a budget of more than a cache holds")
    n, budget, page = 100, 600000, 16
    g = torch.Generator().manual_seed(79)
    k = torch.randn((16, page, 1, 64), generator=g).to(BF).cuda()
    v = torch.randn((16, page, 1, 64), generator=g).to(BF).cuda()
    w = torch.rand((16, 1, page), generator=g).cuda()
    k0, v0, w0 = k.clone(), v.clone(), w.clone()
    table = torch.tensor([[9, 4, 1, 14, 6, 0, 11]], dtype=torch.int32).cuda()
    new = torch.tensor([[2, 3, 5, 7, 8, 10, 12]], dtype=torch.int32).cuda()
    kept, lens = gm.keops_cache_evict(k, v, w, table, torch.tensor([n], dtype=torch.int32).cuda(), new, budget)
    torch.cuda.synchronize()
    assert lens.item() == n and torch.equal(kept[0, 0, :n].cpu(), torch.arange(n, dtype=torch.int32)) and bool((kept[0, 0, n:] == -1).all())
    for pool, old in ((k, k0), (v, v0)):
        got, want = (p[t[0].long()].reshape(-1, 64)[:n] for p, t in ((pool, new), (old, table)))
        assert torch.equal(got, want)
    assert torch.equal(w[new[0].long()].reshape(-1)[:n], w0[table[0].long()].reshape(-1)[:n])


@pytest.mark.parametrize("dim,dtype,cache", [(64, BF, BF), (96, FP, E4), (128, BF, BF), (256, FP, FP)])
@pytest.mark.parametrize("new,heads", [(1, 1), (1, 5), (3, 5), (2, 16)])
def test_many_parts(dim, dtype, cache, new, heads):
    """One head over many work-groups: joined by columns, and its rows' lse by many lanes."""
    say(f"many parts, dim {dim}, {dtype}, {cache}, {new} x {heads} rows")
    b = ref.Batch(83, [27000, 300], [new, 1], heads, 1, dim, 64, dtype, cache)
    b.weights = torch.zeros((b.P, 1, 64))
    check_attention(b)
