"""Calls of the paged cache's operators as programs make them: function transforms, other streams, tables with
holes, bounds far from the lengths.  Against the plain 64-bit forms of paged_reference.py, with its bounds."""
from __future__ import annotations

import pytest
import torch

import paged_reference as ref
from test_gpu_paged import BF, E4, FP, close, put, say, verify_case

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import geometric_map_reduce_amd as gm


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def test_batched_tensors_are_refused():
    """A tensor that torch.vmap batches has no memory of its own: an error in Python, and the calls go on working."""
    say("torch.vmap over q, and over k and v")
    b = ref.Batch(1, [20], [2], 4, 2, 64, 16, junk=0.0)
    q, k, v, table, lens, starts = (put(t) for t in (b.q, b.k, b.v, b.table, b.lens_t(), b.starts))
    want = gm.keops_paged_attention(q, k, v, table, lens, starts, 2, 20)
    rows = q[:, :2].contiguous()
    with pytest.raises((RuntimeError, ValueError)):
        torch.vmap(lambda t: gm.keops_paged_attention(t, k, v, table, lens, starts, 2, 20)[0])(torch.stack([q, q]))
    with pytest.raises((RuntimeError, ValueError)):
        torch.vmap(lambda t: (gm.keops_cache_append(t, t, k, v, table, lens, starts), t)[1])(torch.stack([rows, rows]))
    got = gm.keops_paged_attention(q, k, v, table, lens, starts, 2, 20)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# ---- eviction from tables with holes

def evict_reference(b, new_table, budget, sink, recent):
    """From the definition: of the slots that are there the ones among the first `sink` and the last `recent`, and the
    heaviest of the others (NaN above all; equal weights: the lower slot), `budget` in all, in their order."""
    S, H = len(b.lens), b.kv
    kept, lens = torch.full((S, H, budget), -1, dtype=torch.int32), torch.zeros(S, dtype=torch.int32)
    k, v, w = b.k.clone(), b.v.clone(), b.weights.clone()
    for s, n in enumerate(b.lens):
        there = [j for j in range(n) if 0 <= b.table[s, j // b.page].item() < b.P]
        lens[s] = min(budget, len(there))
        for h in range(H):
            def rank(j):
                x = b.weights[b.table[s, j // b.page].item(), h, j % b.page].item()
                if j < sink or j >= n - recent:
                    return (0, 0.0, j)
                return (1, 0.0, j) if x != x else (2, -x, j)
            for r, j in enumerate(sorted(sorted(there, key=rank)[:budget])):
                kept[s, h, r] = j
                pg, to = b.table[s, j // b.page].item(), new_table[s, r // b.page].item()
                k.view(torch.uint8)[to, r % b.page, h] = b.k.view(torch.uint8)[pg, j % b.page, h]
                v.view(torch.uint8)[to, r % b.page, h] = b.v.view(torch.uint8)[pg, j % b.page, h]
                w[to, h, r % b.page] = b.weights[pg, h, j % b.page]
    return kept, lens, k, v, w


# lens, page, cache, budget, sink, recent, the pages of the table that are missing
HOLES = [
    ([100, 33], 16, BF, 200, 4, 20, [(0, 2), (1, 0)]),                     # all kept but for the holes
    ([100, 90], 16, BF, 60, 20, 30, [(0, 0), (0, 6), (1, 1), (1, 5)]),     # holes among the first and the last
    ([100, 40], 16, FP, 70, 0, 0, [(0, 1), (0, 3), (0, 4), (1, 0), (1, 1), (1, 2)]),   # fewer there than the budget; none at all
    ([64, 64], 6, E4, 50, 7, 9, [(0, 0), (0, 1), (1, 10)]),
    ([40], 1, BF, 35, 3, 3, [(0, 0), (0, 39), (0, 20)]),
    ([9000], 16, BF, 4000, 10, 1000, [(0, 0), (0, 300), (0, 562)]),
    ([40000], 64, BF, 39990, 4, 100, [(0, 1), (0, 624)]),                  # longer than what LDS holds; fewer there than the budget
    ([40000], 24, BF, 500, 30, 100, [(0, 0), (0, 1666)]),
]


@pytest.mark.parametrize("lens,page,cache,budget,sink,recent,missing", HOLES)
@pytest.mark.parametrize("ties", [False, True])
def test_eviction_leaves_out_absent_slots(lens, page, cache, budget, sink, recent, missing, ties):
    """An absent slot is not kept, and nothing of what the new pages held before is seen afterwards."""
    say(f"eviction with holes, {lens} page {page} {cache} budget {budget} sink {sink} recent {recent} missing {missing} ties {ties}")
    H, dim, S = (2 if lens[0] < 1000 else 1), 64, len(lens)
    more = sum(-(-min(n, budget) // page) for n in lens)
    b = ref.Batch(89, lens, [0] * S, H, H, dim, page, FP if cache == FP else BF, cache, spare=more + 1)
    b.weights = torch.rand((b.P, H, page), generator=b.gen)
    if ties:
        b.weights = (b.weights * 3).floor() / 2
        b.weights.view(-1)[::13] = float("nan")
        b.weights.view(-1)[::17] = float("inf")
    for n, (s, at) in enumerate(missing):
        b.table[s, at] = (-1, b.P, 2 ** 31 - 1)[n % 3]
    new = torch.full((S, max(-(-min(n, budget) // page) for n in lens)), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(lens):
        u = -(-min(n, budget) // page)
        new[s, :u] = b.free[at:at + u]
        at += u
    kp, vp, wp = put(b.k), put(b.v), put(b.weights)
    kept, nl = gm.keops_cache_evict(kp, vp, wp, put(b.table), put(b.lens_t()), put(new), budget, sink=sink, recent=recent)
    torch.cuda.synchronize()
    rkept, rl, rk, rv, rw = evict_reference(b, new, budget, sink, recent)
    for name, got, want in (("lens", nl, rl), ("kept", kept, rkept), ("keys", kp, rk), ("values", vp, rv), ("weights", wp, rw)):
        same = torch.equal(got.cpu().view(torch.uint8), want.view(torch.uint8))
        assert same, name
    # a token of each sequence over what is left: the pools' other rows hold NaN
    b.table, b.lens, b.new, b.k, b.v = new, rl.tolist(), [1] * S, rk, rv
    b.T, b.starts = S, torch.arange(S + 1, dtype=torch.int32)
    b.q = (torch.randn((S, H, dim), generator=b.gen) * 2).to(b.dtype)
    out, lse = gm.keops_paged_attention(put(b.q), kp, vp, put(new), nl, put(b.starts), 1, max(b.lens), k_scale=put(b.k_scale),
                                        v_scale=put(b.v_scale))
    o, z, _, ot, zt, _ = ref.attention(b)
    close(lse.cpu(), z, zt, "lse")
    close(out.cpu(), o, ot, "out")


# ---- streams

@pytest.mark.parametrize("handle", [False, True])
def test_outputs_of_another_stream_are_its_own(handle):
    """A block of the output's size is free in the current stream's pool, with a write to it still queued there."""
    say(f"outputs of another stream, its handle {handle}")
    b = ref.Batch(19, [500, 300], [1, 1], 8, 2, 128, 16, junk=0.0)
    b.weights = torch.rand((b.P, 2, 16), generator=b.gen)
    args = [put(t) for t in (b.q, b.k, b.v, b.table, b.lens_t(), b.starts)]
    free = torch.arange(b.P, b.P + 40, dtype=torch.int32)[None].repeat(2, 1)         # pages that are not there: nothing moves
    ver = [put(t) for t in verify_case(5, 2, 3, 5000)]
    w = put(b.weights)

    def calls(s):
        return (*gm.keops_paged_attention(*args, 1, 500, stream=s),
                *gm.keops_cache_evict(args[1], args[2], w, args[3], args[4], free.cuda(), 64, recent=9, stream=s),
                *gm.keops_verify_draft(*ver, stream=s))
    want = calls(None)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)                       # 8 ms of the current stream, or more
    for t in want:
        x = torch.full_like(t, 77)                      # queued behind it
        del x
    got = calls(st.cuda_stream if handle else st)
    st.synchronize()
    on_time = [t.clone() for t in got]                  # read behind the sleep and the writes
    torch.cuda.synchronize()
    for x, y in zip(on_time, want):
        assert torch.equal(x, y)


def test_capture_of_the_stream_that_is_given():
    """The workspace of a call on a captured stream is the graph's, whichever stream is current."""
    say("a captured stream that is not the current one")
    b = ref.Batch(23, [900, 300], [1, 1], 8, 2, 128, 16, junk=0.0)
    args = [put(t) for t in (b.q, b.k, b.v, b.table, b.lens_t(), b.starts)]
    want = gm.keops_paged_attention(*args, 1, 900)
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        with torch.cuda.stream(torch.cuda.default_stream()):
            out, lse = gm.keops_paged_attention(*args, 1, 900, stream=side)
    for _ in range(3):
        out.zero_()
        lse.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
        gm.keops_paged_attention(*args, 1, 900)


# ---- starts outside the tokens

@pytest.mark.parametrize("starts,tokens,lens,want", [
    ([0, 5], 3, [10], [(0, 7, 0), (0, 8, 1), (0, 9, 2)]),
    ([-4, 2], 5, [10], [(0, 8, 0), (0, 9, 1)]),
    ([3, 9, 20], 6, [10, 12], [(0, 7, 3), (0, 8, 4), (0, 9, 5)]),
    ([0, 2, 2 ** 31 - 1], 4, [2, 7], [(0, 0, 0), (0, 1, 1), (1, 5, 2), (1, 6, 3)]),
    ([0, 9], 4, [3], [(0, 0, 1), (0, 1, 2), (0, 2, 3)]),
])
@pytest.mark.parametrize("dtype,cache", [(BF, BF), (FP, E4)])
def test_append_cuts_starts_as_attention_does(starts, tokens, lens, want, dtype, cache):
    """Starts outside [0, tokens] are cut to them: (sequence, slot, token) of each row that is written; attention of the
    same call sees each token in that slot."""
    say(f"append, starts {starts} of {tokens} tokens, {dtype} {cache}")
    S = len(lens)
    b = ref.Batch(97, lens, [0] * S, 2, 2, 64, 4, dtype, cache, junk=0.0)
    b.weights = torch.rand((b.P, 2, 4), generator=b.gen) + 1
    rows = (torch.randn((tokens, 2, 64), generator=b.gen) * 2).to(dtype)
    b.starts = torch.tensor(starts, dtype=torch.int32)
    rk, rv, rw = b.k.clone(), b.v.clone(), b.weights.clone()
    for s, j, t in want:
        pg = b.table[s, j // 4].item()
        for h in range(2):
            for pool, scale in ((rk, b.k_scale), (rv, b.v_scale)):
                x = rows[t, h] if scale is None else (rows[t, h].float() / scale[h]).clamp(-448, 448)
                pool.view(torch.uint8)[pg, j % 4, h] = x.to(cache).view(torch.uint8)
        rw[pg, :, j % 4] = 0.0
    kp, vp, wp, k = put(b.k), put(b.v), put(b.weights), put(rows)
    gm.keops_cache_append(k, k, kp, vp, put(b.table), put(b.lens_t()), put(b.starts), weights=wp, k_scale=put(b.k_scale),
                          v_scale=put(b.v_scale))
    torch.cuda.synchronize()
    for name, got, rest in (("keys", kp, rk), ("values", vp, rv), ("weights", wp, rw)):
        same = torch.equal(got.cpu().view(torch.uint8), rest.view(torch.uint8))
        assert same, name
    # a window of one slot: each token gets the value of its own
    out, _ = gm.keops_paged_attention(k, kp, vp, put(b.table), put(b.lens_t()), put(b.starts), tokens, 16, window=1, k_scale=put(b.k_scale),
                                      v_scale=put(b.v_scale))
    for s, j, t in want:
        v, _ = b.rows(rv, b.v_scale, s, 0, lens[s])
        assert (out[t, 0].double().cpu() - v[j]).abs().max() <= torch.finfo(dtype).eps * v[j].abs().max(), (s, j, t)


# ---- bounds far above the lengths, with weights

def workspace(S, H, rows, dim, pages, page, max_q, max_len):
    """What a call's workspace takes: nothing is launched, and no address read."""
    import ctypes

    from geometric_map_reduce_amd.paged import _CACHE
    row = H * dim
    c = _CACHE.pack(1 << 44, 2 << 44, 3 << 44, 0, 0, page * row, row, dim, pages, 4 << 44, 8192, 5 << 44, page, H, dim, 0, 8192, S)
    n = ctypes.c_int64(0)
    rc = gm.lib().keops_paged_attention_workspace(c, 0, H * rows // max_q, S * max_q, max_q, max_len, 0, ctypes.byref(n))
    assert rc == 0
    return n.value


def test_plans_stay_below_the_threads_of_a_launch():
    """Fewer than 2^32: refused, or with fewer parts."""
    say("plans of many work-groups")
    import ctypes

    from geometric_map_reduce_amd.paged import _CACHE

    def plan(S, H, heads, tokens, max_q, max_len, weights=0, dim=64):
        row = H * dim
        c = _CACHE.pack(1 << 44, 2 << 44, weights, 0, 0, 16 * row, row, dim, 100, 4 << 44, 8192, 5 << 44, 16, H, dim, 0, 8192, S)
        n = ctypes.c_int64(0)
        return gm.lib().keops_paged_attention_workspace(c, 0, heads, tokens, max_q, max_len, 0, ctypes.byref(n)), n.value
    assert plan(1 << 20, 16, 16, 1 << 20, 1, 100) == (-2, 0)              # a work-group to each of 2^24 heads
    assert plan((1 << 20) - 1, 16, 16, 1 << 20, 1, 100) == (0, 0)
    # 2^27 rows in the token arrays, 64 of them in the one sequence: no parts that a join would look through
    assert plan(1, 8, 8, 1 << 24, 64, 20000, dim=256) == (0, 0)
    assert plan(1, 8, 8, 64, 64, 20000, dim=256)[1] > 0
    assert plan(1, 8, 8, 64, 64, 0, weights=3 << 44) == (0, 0)              # no slots: no work-groups to share rows


def test_kept_scores_do_not_outgrow_the_cache():
    say("workspace of steps with weights")
    # one long conversation among short ones: 2.1 GB of scores for 0.8 GB of keys and values
    assert workspace(64, 8, 8, 128, 194000 // 16, 16, 1, 131072) < 1e8
    # more than 4 GB, whatever the cache
    assert workspace(64, 8, 32, 128, 64 * 8192, 16, 4, 131072) < 1e8
    # as large as the lengths may want: kept
    assert workspace(64, 8, 8, 128, 64 * 8192, 16, 1, 131072) > 4 * 64 * 8 * 8 * 131072
    assert workspace(32, 8, 4, 128, 32 * 313, 16, 1, 8000) > 4 * 32 * 8 * 4 * 8000


@pytest.mark.parametrize("new,dtype,cache", [(1, BF, BF), (2, FP, FP), (2, BF, E4)])
def test_weights_under_far_bounds(new, dtype, cache):
    """Weights by the column sums instead of kept scores, of few rows."""
    say(f"weights under far bounds, {new} new, {dtype} {cache}")
    b = ref.Batch(101, [300, 77, 0, 2000], [new, 1, 0, new], 8, 2, 128, 24, dtype, cache)
    b.weights = torch.rand((b.P, 2, 24), generator=b.gen)
    w = put(b.weights)
    out, lse = gm.keops_paged_attention(put(b.q), put(b.k), put(b.v), put(b.table), put(b.lens_t()), put(b.starts), new, 1 << 23,
                                        weights=w, decay=0.5, k_scale=put(b.k_scale), v_scale=put(b.v_scale))
    o, z, ww, ot, zt, wt = ref.attention(b, 0.5)
    close(lse.cpu(), z, zt, "lse")
    close(out.cpu(), o, ot, "out")
    close(w.cpu(), ww, wt, "weights")


# ---- verification

@pytest.mark.parametrize("given", [False, True])
def test_tokens_outside_the_vocabulary_are_refused_whatever_the_number(given):
    say(f"verification of tokens outside the vocabulary, draft {given}")
    target, draft, tokens, counts, ua, us = verify_case(103, 6, 3, 257)
    counts[:] = 3
    for s, x in enumerate((-1, 257, 2 ** 31 - 1, -2 ** 31)):
        tokens[s, s % 3] = x
        ua[s] = -0.5
    out, acc = gm.keops_verify_draft(put(target), put(draft) if given else None, put(tokens), put(counts), put(ua), put(us))
    ro, ra = ref.verify(target, draft if given else None, tokens, counts, ua, us)
    assert acc.tolist() == ra.tolist() and out.tolist() == ro.tolist()


# ---- no new tokens

@pytest.mark.parametrize("tokens,max_q", [(0, 0), (0, 1), (0, 500), (3, 0)])
@pytest.mark.parametrize("decay", [0.0, 0.5])
@pytest.mark.parametrize("dtype,cache", [(BF, BF), (FP, E4)])
def test_weights_without_new_tokens(tokens, max_q, decay, dtype, cache):
    """A call in which no sequence has a token that counts gives no slot anything: the weights become decay * old."""
    say(f"weights, {tokens} tokens, max_q {max_q}, decay {decay}, {cache}")
    b = ref.Batch(107, [300, 0, 20], [tokens, 0, 0], 8, 2, 64, 16, dtype, cache, junk=0.0)
    b.weights = torch.rand((b.P, 2, 16), generator=b.gen)
    w = put(b.weights)
    out, lse = gm.keops_paged_attention(put(b.q), put(b.k), put(b.v), put(b.table), put(b.lens_t()), put(b.starts), max_q, 300,
                                        weights=w, decay=decay, k_scale=put(b.k_scale), v_scale=put(b.v_scale))
    torch.cuda.synchronize()
    assert out.shape == (tokens, 8, 64) and lse.shape == (tokens, 8)
    want = b.weights.clone()
    for s, n in ((0, 300), (2, 20)):
        for j in range(n):
            want[b.table[s, j // 16].item(), :, j % 16] *= decay
    assert torch.equal(w.cpu(), want)


def test_the_default_stream_by_its_handle():
    say("the default stream by its handle, another one current")
    b = ref.Batch(19, [500, 300], [1, 1], 8, 2, 128, 16, junk=0.0)
    args = [put(t) for t in (b.q, b.k, b.v, b.table, b.lens_t(), b.starts)]
    want = gm.keops_paged_attention(*args, 1, 500)
    torch.cuda.synchronize()
    for current in (torch.cuda.default_stream(), torch.cuda.Stream()):
        with torch.cuda.stream(current):
            got = gm.keops_paged_attention(*args, 1, 500, stream=0)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
