"""Refusals of the paged cache and of draft verification, on the host: the C ABI rejects what it cannot
take before any HIP call, and the binding names what is wrong with a tensor."""
import ctypes
import os

import pytest
import torch

import geometric_map_reduce_amd as gm
from geometric_map_reduce_amd import binding
from geometric_map_reduce_amd.paged import _CACHE

A, B, C, D, E, F, G = (0x10000000 * (i + 1) for i in range(7))    # never dereferenced: validation fails first


class _Cache(ctypes.Structure):
    """keops_cache_t as the header declares it."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("k_pages", "v_pages", "weights", "k_scale", "v_scale")] + \
        [(n, ctypes.c_int64) for n in ("page_stride", "slot_stride", "head_stride", "pages")] + \
        [("page_table", ctypes.c_void_p), ("table_stride", ctypes.c_int64), ("lens", ctypes.c_void_p)] + \
        [(n, ctypes.c_int32) for n in ("page_size", "heads", "dim", "type", "table_width", "seqs")]


def test_binding_packs_the_structure():
    vals = list(range(1, 19))
    c = _Cache.from_buffer_copy(_CACHE.pack(*vals))
    assert _CACHE.size == ctypes.sizeof(_Cache) and [getattr(c, n) for n, _ in _Cache._fields_] == vals


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(binding.LIB_PATH):
        pytest.skip("library not built")
    return binding.lib()


def cache(**kw):
    c = _Cache()
    c.k_pages, c.v_pages, c.page_table, c.lens = A, B, C, D
    c.page_stride, c.slot_stride, c.head_stride = 16 * 2 * 64, 2 * 64, 64
    c.pages, c.page_size, c.heads, c.dim, c.type = 10, 16, 2, 64, 0
    c.table_stride, c.table_width, c.seqs = 4, 4, 3
    for k, v in kw.items():
        setattr(c, k, v)
    return c


BAD_CACHES = [
    (dict(pages=-1), -1), (dict(page_size=0), -1), (dict(heads=0), -1), (dict(dim=0), -1), (dict(seqs=-1), -1),
    (dict(table_width=-1), -1), (dict(type=3), -1), (dict(type=-1), -1), (dict(type=2), -1),       # scales missing
    (dict(k_pages=None), -1), (dict(v_pages=None), -1), (dict(lens=None), -1), (dict(page_table=None), -1),
    (dict(k_pages=A + 8), -1), (dict(lens=D + 2), -1), (dict(weights=E + 1), -1),
    (dict(slot_stride=129), -1), (dict(page_stride=-64), -1), (dict(head_stride=4), -1),
    (dict(dim=80), -2), (dict(dim=512), -2), (dict(pages=1 << 31), -2),
]


def call_append(L, c, k=E, v=F, ks=128, vs=128, type=0, starts=G, tokens=5):
    return L.keops_cache_append(None if c is None else ctypes.addressof(c), k, v, ks, vs, type, starts, tokens, None)


def call_attend(L, c, q=E, qs=256, type=0, heads=4, starts=G, tokens=5, max_q=2, max_len=64, scale=0.1, window=0, decay=0.0,
                out=0x80000000, lse=0x90000000, ws=None, nbytes=0):
    return L.keops_paged_attention(None if c is None else ctypes.addressof(c), q, qs, type, heads, starts, tokens, max_q, max_len,
                                   scale, window, decay, out, lse, ws, nbytes, None)


def call_evict(L, c, new=E, stride=4, width=4, budget=20, sink=1, recent=2, kept=F, lens=G):
    return L.keops_cache_evict(None if c is None else ctypes.addressof(c), new, stride, width, budget, sink, recent, kept, lens, None)


@pytest.mark.parametrize("kw,rc", BAD_CACHES)
def test_bad_caches(L, kw, rc):
    c = cache(**kw)
    assert call_append(L, c) == rc
    assert call_attend(L, c) == rc
    if "type" not in kw or kw["type"] != 2:
        if c.weights is None:
            c.weights = 0xA0000000
        assert call_evict(L, c) == rc


def test_append_refusals(L):
    assert call_append(L, None) == -1
    for kw in (dict(k=None), dict(v=None), dict(k=E + 2), dict(ks=129), dict(vs=-128), dict(type=2), dict(type=1), dict(starts=None),
               dict(starts=G + 1), dict(tokens=-1), dict(k=A), dict(v=B + 16)):
        assert call_append(L, cache(), **kw) == -1, kw
    assert call_append(L, cache(), tokens=1 << 31) == -2
    assert call_append(L, cache(), tokens=0, k=None, v=None, starts=None) == 0
    assert call_append(L, cache(seqs=0, lens=None, page_table=None), starts=None) == 0


def test_attention_refusals(L):
    assert call_attend(L, None) == -1
    for kw in (dict(q=None), dict(out=None), dict(lse=None), dict(q=E + 4), dict(out=0x80000002), dict(lse=0x90000001),
               dict(qs=257), dict(type=2), dict(type=1), dict(heads=3), dict(heads=0), dict(starts=None), dict(tokens=-1),
               dict(max_q=-1), dict(max_len=-1), dict(window=-1), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(decay=float("nan")), dict(out=E), dict(out=A), dict(lse=E), dict(lse=0x80000000), dict(ws=0xB0000080, nbytes=64),
               dict(ws=0xB0000000, nbytes=-1)):
        assert call_attend(L, cache(), **kw) == -1, kw
    assert call_attend(L, cache(weights=0x80000000)) == -1       # out over the weights
    assert call_attend(L, cache(pages=0, k_pages=None, v_pages=None)) == -1
    assert call_attend(L, cache(), tokens=1 << 31, out=1 << 50, lse=1 << 52, q=1 << 54) == -2
    assert call_attend(L, cache(), max_q=1 << 30) == -2
    assert call_attend(L, cache(), max_len=(1 << 30) + 1) == -2
    assert call_attend(L, cache(), tokens=0, q=None, out=None, lse=None, starts=None) == 0
    assert call_attend(L, cache(), max_q=0) == 0
    n = ctypes.c_int64(7)
    assert L.keops_paged_attention_workspace(ctypes.addressof(cache()), 0, 4, 0, 2, 64, 0, ctypes.byref(n)) == 0 and n.value == 0
    assert L.keops_paged_attention_workspace(ctypes.addressof(cache()), 0, 3, 5, 2, 64, 0, ctypes.byref(n)) == -1


def test_evict_refusals(L):
    ok = cache(weights=0xA0000000)
    assert call_evict(L, None) == -1
    for kw in (dict(new=None), dict(kept=None), dict(lens=None), dict(kept=F + 2), dict(budget=0), dict(sink=-1), dict(recent=-1),
               dict(sink=15, recent=6), dict(width=1), dict(lens=D), dict(kept=D), dict(kept=A)):
        assert call_evict(L, ok, **kw) == -1, kw
    assert call_evict(L, cache()) == -1                          # no weights
    assert call_evict(L, cache(weights=0xA0000000, table_width=1 << 28), width=1 << 28) == -2
    far = dict(weights=1 << 50, k_pages=1 << 51, v_pages=1 << 52)
    assert call_evict(L, cache(pages=1 << 30, **far)) == -2            # weight numbers past 32 bits
    assert call_evict(L, cache(weights=0xA0000000, seqs=0, lens=None, page_table=None), new=None, kept=None, lens=None) == 0


def test_verify_refusals(L):
    def call(target=A, draft=B, tokens=C, counts=D, ua=E, us=F, S=2, K=3, V=100, out=G, acc=0x90000000, ws=None, nbytes=0):
        return L.keops_verify_draft(target, draft, tokens, counts, ua, us, S, K, V, out, acc, ws, nbytes, None)
    for kw in (dict(target=None), dict(tokens=None), dict(counts=None), dict(ua=None), dict(us=None), dict(out=None), dict(acc=None),
               dict(S=-1), dict(K=-1), dict(V=0), dict(target=A + 2), dict(out=G + 1), dict(out=A), dict(acc=G), dict(out=C),
               dict(acc=D), dict(ws=0xB0000001, nbytes=64), dict(ws=0xB0000000, nbytes=-1)):
        assert call(**kw) == -1, kw
    assert call(V=(1 << 30) + 1) == -2
    n = ctypes.c_int64(7)
    assert L.keops_verify_draft_workspace(5, 3, 131072, ctypes.byref(n)) == 0 and n.value == 5 * 64 * 16
    assert L.keops_verify_draft_workspace(-1, 3, 10, ctypes.byref(n)) == -1
    assert call(S=0, target=None, tokens=None, counts=None, ua=None, us=None, out=None, acc=None) == 0


def test_binding_refuses_host_tensors():
    k = torch.zeros((4, 16, 2, 64), dtype=torch.bfloat16)
    i = torch.zeros((1,), dtype=torch.int32)
    with pytest.raises(ValueError, match="k_pages"):
        gm.keops_paged_attention(torch.zeros((1, 2, 64), dtype=torch.bfloat16), k, k.clone(), torch.zeros((1, 4), dtype=torch.int32), i,
                                 torch.zeros((2,), dtype=torch.int32), 1, 1)
    with pytest.raises(TypeError, match="lens"):
        gm.keops_cache_evict(k, k, None, None, None, None, 4)
    with pytest.raises(TypeError, match="target"):
        gm.keops_verify_draft(None, None, None, None, None, None)
    with pytest.raises(ValueError, match="target"):
        gm.keops_verify_draft(torch.zeros((1, 2, 8)), None, torch.zeros((1, 1), dtype=torch.int32), None, None, None)


def test_evict_refuses_more_heads_of_sequences_than_a_grid_has(L):
    far = dict(k_pages=1 << 51, v_pages=1 << 52, weights=1 << 53)
    c = cache(seqs=40000, heads=65535, pages=10, page_size=1, table_width=1, **far)
    assert call_evict(L, c, budget=1, sink=0, recent=0, kept=1 << 54, lens=1 << 55) == -2


def test_short_way_hands_back_what_it_does_not_take(L):
    """Nothing that is no plain tensor on the current device is taken, and no argument raises or ends the process."""
    from geometric_map_reduce_amd import paged
    short = paged._native()
    x, i = torch.zeros((1, 2, 64), dtype=torch.bfloat16), torch.zeros((2,), dtype=torch.int32)
    k = torch.zeros((4, 16, 2, 64), dtype=torch.bfloat16)
    good = [x, x, k, k, None, i[None], i[:1], None, None, i]
    for at in range(len(good)):
        for bad in (None, 3, "k", [x], object(), torch.nn.Parameter(x), x.to("meta"), torch.zeros((0,)), i):
            a = list(good)
            a[at] = bad
            assert short.append(*a) is None
            assert short.attention(a[0], *a[2:], 1, 16, None, 0, 0.0, None, None) is None
            assert short.evict(*a[2:8], None, i[None], 4, 0, 0, None, None) is None
            assert short.verify(*a[:6], None, None) is None
    assert short.append() is None and short.append(*good, 1) is None and short.attention(*good) is None
    assert short.evict() is None and short.verify() is None


def test_calls_of_more_threads_than_a_launch_has_are_refused(L):
    """A launch has fewer than 2^32 threads."""
    far = dict(k_pages=1 << 51, v_pages=1 << 52, weights=1 << 53)
    c = cache(weights=1 << 53)
    assert call_append(L, c, k=1 << 54, v=1 << 55, tokens=1 << 28) == -2           # 16 pieces a token
    evict = dict(kept=1 << 54, lens=1 << 55, sink=0, recent=0)
    assert call_evict(L, cache(seqs=4096, heads=16, **far), budget=8192, **evict) == -2
    assert call_evict(L, cache(seqs=65536, heads=64, **far), budget=1, **evict) == -2
    n = ctypes.c_int64(7)
    assert L.keops_verify_draft_workspace(1 << 24, 0, 1, ctypes.byref(n)) == -2
    assert L.keops_verify_draft_workspace(1 << 18, 0, 131072, ctypes.byref(n)) == -2
    assert L.keops_verify_draft(1 << 54, None, None, D, None, F, 1 << 24, 0, 1, 1 << 55, 1 << 56, None, 0, None) == -2
