"""Rotary positions, the rotating append, reading slots back and the adjustment of logits on a host without a GPU: what
the C ABI and the binding refuse, the structures that the binding packs, the frequencies, and the compiled way from tensors
(``native/step_call.cpp``) over a stand-in for the library (``tests/step_call_stub.cpp``)."""
import ctypes
import importlib.util
import math
import os
import subprocess
import sys
import sysconfig

import pytest
import torch

import geometric_map_reduce_amd as gm
from geometric_map_reduce_amd import binding, paged, step
from test_paged_host import A, B, C, D, E, F, G, _Cache, cache, call_append, call_attend, call_evict

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
H1, H2, H3 = 0x100000000, 0x200000000, 0x300000000       # never dereferenced


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(binding.LIB_PATH):
        pytest.skip("library not built")
    return binding.lib()


class _Rotary(ctypes.Structure):
    """keops_rotary_t as the header declares it."""
    _fields_ = [("freqs", ctypes.c_void_p), ("factor", ctypes.c_double), ("pairs", ctypes.c_int32), ("interleaved", ctypes.c_int32)]


class _Rules(ctypes.Structure):
    """keops_logit_rules_t as the header declares it."""
    _fields_ = [("starts", ctypes.c_void_p), ("text", ctypes.c_void_p), ("text_stride", ctypes.c_int64)] + \
        [(n, ctypes.c_void_p) for n in ("lens", "prompt_lens", "repetition", "presence", "frequency", "bias_tokens", "bias", "mask")] + \
        [("mask_stride", ctypes.c_int64)] + [(n, ctypes.c_int32) for n in ("seqs", "text_width", "biases")]


def test_binding_packs_the_structures():
    r = _Rotary.from_buffer_copy(step._ROTARY.pack(1, 2.5, 3, 4))
    assert step._ROTARY.size == ctypes.sizeof(_Rotary) and [getattr(r, n) for n, _ in _Rotary._fields_] == [1, 2.5, 3, 4]
    vals = list(range(1, 16))
    r = _Rules.from_buffer_copy(step._RULES.pack(*vals))
    assert step._RULES.size == ctypes.sizeof(_Rules) and [getattr(r, n) for n, _ in _Rules._fields_] == vals


def test_structures_have_the_size_that_c_gives_them(tmp_path):
    src = tmp_path / "s.c"
    src.write_text('#include "keops_mi355x.h"\n#include <stdio.h>\n#include <stddef.h>\nint main(void) {\n'
                   '  printf("%zu %zu %zu %zu %zu\\n", sizeof(keops_cache_t), offsetof(keops_cache_t, k_powers), sizeof(keops_rotary_t),\n'
                   '         sizeof(keops_logit_rules_t), offsetof(keops_logit_rules_t, seqs));\n  return 0;\n}\n')
    exe = str(tmp_path / "s")
    res = subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o", exe],
                         capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    got = [int(x) for x in subprocess.run([exe], capture_output=True, text=True).stdout.split()]
    assert got == [ctypes.sizeof(_Cache), _Cache.k_scale.offset, ctypes.sizeof(_Rotary), ctypes.sizeof(_Rules), _Rules.seqs.offset]


# ---- the frequencies

def test_frequencies():
    f = gm.keops_rotary_frequencies(8, 100.0)
    assert f.dtype == torch.float64 and torch.allclose(f, torch.tensor([1, 100 ** -0.25, 0.1, 100 ** -0.75], dtype=torch.float64), rtol=1e-15)
    assert torch.allclose(gm.keops_rotary_frequencies(8, 100.0, "linear", 4.0), f / 4, rtol=1e-15)
    b = gm.keops_rotary_frequencies(8, 100.0, "base", 4.0)
    assert b[0] == 1 and torch.allclose(b[-1], f[-1] / 4, rtol=1e-14) and bool((b[1:-1] < f[1:-1]).all())
    p = gm.keops_rotary_frequencies(64, 10000.0, "parts", 8.0, length=2048, slow=1, fast=32)
    f = gm.keops_rotary_frequencies(64)
    turns = 2048 * f / (2 * math.pi)
    assert torch.equal(p[turns >= 32], f[turns >= 32]) and torch.allclose(p[turns <= 1], f[turns <= 1] / 8, rtol=1e-15)
    mid = (turns > 1) & (turns < 32)
    assert bool(mid.any()) and bool((p[mid] < f[mid]).all()) and bool((p[mid] > f[mid] / 8).all())
    for bad in (dict(dim=7), dict(dim=0), dict(dim=8, base=0.0), dict(dim=8, scaling="other"), dict(dim=8, scaling="parts"),
                dict(dim=8, factor=0.0), dict(dim=2, scaling="base"), dict(dim=8, scaling="parts", length=9, slow=3, fast=3)):
        with pytest.raises(ValueError):
            gm.keops_rotary_frequencies(**bad)


# ---- the C ABI

def rotary(**kw):
    r = _Rotary(freqs=H1, factor=1.0, pairs=16, interleaved=0)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def call_rotary(L, r, x=A, xs=256, type=0, tokens=5, heads=4, dim=64, at=B, inverse=0, out=C, os=256):
    return L.keops_rotary(x, xs, type, tokens, heads, dim, at, None if r is None else ctypes.addressof(r), inverse, out, os, None)


def test_rotary_refusals(L):
    assert call_rotary(L, None) == -1
    for kw in (dict(freqs=None), dict(freqs=H1 + 4), dict(pairs=-1), dict(pairs=33), dict(factor=float("nan")), dict(factor=float("inf"))):
        assert call_rotary(L, rotary(**kw)) == -1, kw
    for kw in (dict(x=None), dict(out=None), dict(at=None), dict(x=A + 1), dict(out=C + 1), dict(at=B + 2), dict(type=2), dict(type=4),
               dict(type=-1), dict(type=3, x=A + 2), dict(tokens=-1), dict(heads=-1), dict(dim=0), dict(xs=-1), dict(os=255), dict(xs=1 << 41),
               dict(out=A + 2), dict(out=A, os=300), dict(out=B), dict(out=H1)):
        assert call_rotary(L, rotary(), **kw) == -1, kw
    assert call_rotary(L, rotary(), dim=65537, os=1 << 30, out=1 << 50) == -2 and call_rotary(L, rotary(), heads=65536, os=1 << 30, out=1 << 50) == -2
    assert call_rotary(L, rotary(), tokens=1 << 31, out=1 << 50, x=1 << 52, at=1 << 54) == -2
    assert call_rotary(L, rotary(pairs=8193), dim=32768, os=1 << 20, out=1 << 50, x=1 << 52) == -2
    assert call_rotary(L, rotary(), tokens=0, x=None, out=None, at=None) == 0
    assert call_rotary(L, rotary(), heads=0, x=None, out=None, at=None) == 0
    # nothing turns, in place: nothing to do
    assert call_rotary(L, rotary(pairs=0, freqs=None), out=A, at=None) == 0


def call_turn(L, c, r, q=E, k=F, v=G, qs=256, ks=128, vs=128, type=0, heads=4, starts=H2, tokens=5, at=None, out=H3, os=256):
    return L.keops_cache_append_rotary(None if c is None else ctypes.addressof(c), q, k, v, qs, ks, vs, type, heads, starts, tokens, at,
                                       None if r is None else ctypes.addressof(r), out, os, None)


def test_append_rotary_refusals(L):
    assert call_turn(L, None, rotary()) == -1 and call_turn(L, cache(), None) == -1
    for kw in (dict(freqs=None), dict(pairs=33), dict(factor=float("inf"))):
        assert call_turn(L, cache(), rotary(**kw)) == -1, kw
    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(q=E + 8), dict(out=H3 + 8), dict(qs=257), dict(os=248), dict(ks=-8),
               dict(type=1), dict(type=2), dict(type=3), dict(type=4), dict(starts=None), dict(starts=H2 + 1), dict(at=H1 + 2), dict(tokens=-1),
               dict(heads=-1), dict(out=E), dict(out=F), dict(out=A), dict(k=A), dict(v=B + 16), dict(q=A), dict(out=H1 - 16)):
        assert call_turn(L, cache(), rotary(), **kw) == -1, kw
    assert call_turn(L, cache(dim=80), rotary()) == -2 and call_turn(L, cache(), rotary(), heads=65536) == -2
    far = dict(q=1 << 50, k=1 << 51, v=1 << 52, out=1 << 53)
    assert call_turn(L, cache(), rotary(), tokens=1 << 31, **far) == -2
    assert call_turn(L, cache(), rotary(), tokens=1 << 25, **far) == -2                 # more threads than a launch has
    assert call_turn(L, cache(), rotary(), tokens=0, q=None, k=None, v=None, out=None, starts=None) == 0
    assert call_turn(L, cache(seqs=0, lens=None, page_table=None), rotary(), starts=None) == 0


def call_read(L, c, k=E, v=F, ks=128, vs=128, type=0, starts=G, tokens=5):
    return L.keops_cache_read(None if c is None else ctypes.addressof(c), k, v, ks, vs, type, starts, tokens, None)


def test_read_refusals(L):
    assert call_read(L, None) == -1
    for kw in (dict(k=None), dict(v=None), dict(k=E + 2), dict(ks=129), dict(vs=-128), dict(ks=120), dict(type=2), dict(type=1), dict(type=4),
               dict(starts=None), dict(starts=G + 1), dict(tokens=-1), dict(k=A), dict(v=B + 16), dict(v=E), dict(v=E + 256, ks=136, vs=136)):
        assert call_read(L, cache(), **kw) == -1, kw
    assert call_read(L, cache(weights=E)) == -1
    assert call_read(L, cache(), k=1 << 50, v=1 << 52, tokens=1 << 31) == -2
    assert call_read(L, cache(), tokens=0, k=None, v=None, starts=None) == 0
    assert call_read(L, cache(seqs=0, lens=None, page_table=None), starts=None) == 0


def four_bit(**kw):
    return cache(**dict(dict(type=4, k_scale=0x90000000, v_scale=0xA0000000, page_stride=16 * 2 * 64, slot_stride=2 * 64, head_stride=64), **kw))


def test_four_bit_caches(L):
    """What the calls over a cache refuse of a 4-bit one; strides count values, two to a byte."""
    for kw in (dict(k_scale=None), dict(v_scale=None), dict(k_scale=0x90000008), dict(v_scale=0xA0000002), dict(slot_stride=2 * 64 + 8),
               dict(head_stride=16), dict(page_stride=-32)):
        c = four_bit(**kw)
        assert call_append(L, c) == -1 and call_attend(L, c) == -1 and call_read(L, c) == -1 and call_turn(L, c, rotary()) == -1, kw
        c.weights = 0xB0000000
        assert call_evict(L, c) == -1, kw
    c = four_bit(pages=1 << 30, k_pages=1 << 50, v_pages=1 << 51, k_scale=1 << 52, v_scale=1 << 53)
    assert call_append(L, c) == -2 and call_attend(L, c) == -2 and call_read(L, c) == -2 and call_turn(L, c, rotary()) == -2
    assert call_append(L, four_bit(), type=4) == -1 and call_attend(L, four_bit(), type=4) == -1
    # the powers are part of the pool: no input or output may lie in them
    assert call_append(L, four_bit(), k=0x90000000) == -1 and call_append(L, four_bit(), v=0xA0000000 + 16) == -1
    assert call_attend(L, four_bit(), out=0xA0000000) == -1 and call_attend(L, four_bit(), lse=0x90000000 + 4) == -1
    assert call_evict(L, four_bit(weights=0xC0000000), kept=0x90000000) == -1
    assert call_read(L, four_bit(), k=0x90000000) == -1 and call_turn(L, four_bit(), rotary(), out=0xA0000000) == -1
    assert call_append(L, cache(type=3)) == -1                # 32 bits are no cache's


def rules(**kw):
    r = _Rules(starts=A, text=B, text_stride=50, lens=C, prompt_lens=D, repetition=E, presence=F, frequency=G, bias_tokens=H1, bias=H2,
               mask=H3, mask_stride=4, seqs=3, text_width=50, biases=6)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def call_logits(L, r, z=0x400000000, stride=100, type=3, rows=5, vocab=100, out=0x500000000, os=100):
    return L.keops_adjust_logits(z, stride, type, rows, vocab, None if r is None else ctypes.addressof(r), out, os, None)


def test_long_lists_of_biases_are_refused(L):
    """Past 2^30 entries a thread's place in the list, half a thousand further each turn, could pass 31 bits."""
    far = dict(bias_tokens=1 << 45, bias=1 << 46, seqs=1)
    for n in ((1 << 30) + 1, (1 << 31) - 1):
        assert call_logits(L, rules(biases=n, **far)) == -2


def test_logits_refusals(L):
    assert call_logits(L, None) == -1
    for kw in (dict(starts=None), dict(lens=None), dict(bias=None), dict(bias_tokens=None), dict(seqs=-1), dict(text_width=-1), dict(biases=-1),
               dict(text_stride=-1), dict(mask_stride=-1), dict(starts=A + 1), dict(text=B + 2), dict(mask=H3 + 3), dict(frequency=G + 1)):
        assert call_logits(L, rules(**kw)) == -1, kw
    for kw in (dict(z=None), dict(out=None), dict(z=0x400000002), dict(out=0x500000001), dict(stride=-1), dict(os=99), dict(type=2), dict(type=4),
               dict(rows=-1), dict(vocab=0), dict(out=0x400000004), dict(out=0x400000000, os=104), dict(out=A), dict(out=B), dict(out=H3),
               dict(out=H2 - 64), dict(out=D)):
        assert call_logits(L, rules(), **kw) == -1, kw
    assert call_logits(L, rules(), rows=1 << 31, z=1 << 50, out=1 << 52) == -2
    assert call_logits(L, rules(), vocab=(1 << 30) + 1, os=1 << 31, z=1 << 50, out=1 << 52) == -2
    assert call_logits(L, rules(), rows=1 << 24, vocab=1 << 20, os=1 << 20, z=1 << 55, out=1 << 58, stride=1 << 20) == -2    # threads of a launch
    assert call_logits(L, rules(), rows=0, z=None, out=None) == 0
    assert call_logits(L, _Rules(), z=None, out=None) == 0


# ---- the binding

def test_binding_names_what_is_wrong():
    bf, i32 = torch.bfloat16, torch.int32
    x, i = torch.zeros((2, 2, 64), dtype=bf), torch.zeros((2,), dtype=i32)
    f = torch.zeros(8, dtype=torch.float64)
    k = torch.zeros((4, 16, 2, 64), dtype=bf)
    with pytest.raises(TypeError, match="x must"):
        gm.keops_rotary(None, i, f)
    with pytest.raises(TypeError, match="positions"):
        gm.keops_rotary(x, None, f)
    with pytest.raises(ValueError, match="x must be"):
        gm.keops_rotary(x, i, f)                         # on the host
    with pytest.raises(ValueError, match="k_pages"):
        gm.keops_cache_append_rotary(x, x, x, k, k.clone(), i[None], i[:1], i, f)
    with pytest.raises(TypeError, match="k_pages"):
        gm.keops_cache_read(None, k, i[None], i[:1], i, 2)
    with pytest.raises(ValueError, match="k_pages"):
        gm.keops_cache_read(k, k.clone(), i[None], i[:1], i, 2)
    with pytest.raises(TypeError, match="logits"):
        gm.keops_adjust_logits(None, i)
    with pytest.raises(ValueError, match="logits"):
        gm.keops_adjust_logits(torch.zeros((2, 8)), i)


@pytest.fixture
def host(monkeypatch):
    """The binding's own checks of host tensors, as if they were on device 0, down to the library."""
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
    for module in (paged, step):
        monkeypatch.setattr(module, "_other", lambda stream, dev: None)
    for module in (step, paged):
        monkeypatch.setattr(module, "_native", lambda: None)
        monkeypatch.setattr(module, "_short", None)
    ran = []
    monkeypatch.setattr(step, "_run", lambda name, *a: ran.append(name))
    return ran


def test_binding_refusals(host):
    bf, i32, f64 = torch.bfloat16, torch.int32, torch.float64
    x, at, f = torch.zeros((2, 2, 64), dtype=bf), torch.zeros(2, dtype=i32), torch.zeros(32, dtype=f64)
    assert gm.keops_rotary(x, at, f).shape == x.shape
    for match, args in (("x must", (x.to(torch.float64), at, f)), ("x must", (x[0], at, f)), ("positions", (x, at.long(), f)),
                        ("positions", (x, at[:1], f)), ("freqs", (x, at, f.float())), ("freqs", (x, at, torch.zeros(33, dtype=f64))),
                        ("freqs", (x, at, f[None])), ("dense", (torch.zeros((2, 64, 2), dtype=bf).transpose(1, 2), at, f)),
                        ("factor", (x, at, f, False, float("nan"))), ("out", (x, at, f, False, 1.0, False, x.float())),
                        ("out", (x, at, f, False, 1.0, False, x[:1]))):
        with pytest.raises(ValueError, match=match):
            gm.keops_rotary(*args)
    pages = torch.zeros((4, 16, 2, 32), dtype=torch.uint8).view(torch.float4_e2m1fn_x2)
    p = torch.zeros((4, 2, 16, 2), dtype=torch.uint8).view(torch.float8_e8m0fnu)
    table, lens, starts = torch.zeros((1, 4), dtype=i32), torch.ones(1, dtype=i32), torch.tensor([0, 2], dtype=i32)
    good = dict(q=x, k=x, v=x.clone(), k_pages=pages, v_pages=pages.clone(), page_table=table, lens=lens, starts=starts, freqs=f, k_scale=p,
                v_scale=p.clone())
    assert gm.keops_cache_append_rotary(**good).shape == x.shape
    for match, kw in (("needs k_scale", dict(k_scale=None)), ("v_scale", dict(v_scale=p[..., :1])), ("k_scale", dict(k_scale=torch.zeros(2))),
                      ("v_pages", dict(v_pages=pages[:3])), ("q must", dict(q=x.to(torch.float16))), ("q must", dict(q=x[:1])),
                      ("v must", dict(v=x.to(torch.float16))), ("positions", dict(positions=at.long())), ("freqs", dict(freqs=f.float())),
                      ("out", dict(out=x.float())), ("starts", dict(starts=at.new_zeros(3)))):
        with pytest.raises(ValueError, match=match):
            gm.keops_cache_append_rotary(**dict(good, **kw))
    cached = {n: good[n] for n in ("k_pages", "v_pages", "page_table", "lens", "starts", "k_scale", "v_scale")}
    k, v = gm.keops_cache_read(**cached, tokens=2)
    assert k.shape == (2, 2, 64) and k.dtype == bf and v.shape == k.shape
    for match, kw in (("dtype", dict(dtype=torch.float32)), ("tokens", dict(tokens=-1)), ("needs k_scale", dict(v_scale=None)),
                      ("out", dict(out=(k, v[:1])))):
        with pytest.raises(ValueError, match=match):
            gm.keops_cache_read(**dict(dict(cached, tokens=2), **kw))
    z = torch.zeros((2, 40))
    rules = dict(starts=starts, tokens=torch.zeros((1, 9), dtype=i32), lens=lens, prompt_lens=lens, repetition=torch.ones(1), presence=torch.ones(1),
                 frequency=torch.ones(1), bias_tokens=torch.zeros((1, 3), dtype=i32), bias=torch.zeros((1, 3)), mask=torch.zeros((2, 2), dtype=i32))
    assert gm.keops_adjust_logits(z, **rules).shape == z.shape
    for match, kw in (("lens", dict(lens=None)), ("need tokens", dict(tokens=None)), ("belong together", dict(bias=None)), ("mask", dict(mask=rules["mask"][:, :1])),
                      ("mask", dict(mask=torch.zeros((1, 2), dtype=i32))), ("repetition", dict(repetition=torch.ones(2))),
                      ("bias_tokens", dict(bias_tokens=torch.zeros((1, 3)))), ("bias", dict(bias=torch.zeros((1, 2)))),
                      ("tokens", dict(tokens=torch.zeros((1, 9)))), ("out", dict(out=z.half())), ("starts", dict(starts=starts[None]))):
        with pytest.raises(ValueError, match=match):
            gm.keops_adjust_logits(z, **dict(rules, **kw))
    with pytest.raises(ValueError, match="contiguous rows"):
        gm.keops_adjust_logits(torch.zeros((40, 2)).T, starts)
    assert host == ["keops_rotary", "keops_cache_append_rotary", "keops_cache_read", "keops_adjust_logits"]


def test_eviction_needs_the_powers_of_a_4_bit_cache(host):
    pages = torch.zeros((4, 16, 2, 32), dtype=torch.uint8).view(torch.float4_e2m1fn_x2)
    i = torch.zeros((1, 4), dtype=torch.int32)
    with pytest.raises(ValueError, match="needs k_scale"):
        gm.keops_cache_evict(pages, pages, torch.zeros((4, 2, 16)), i, i[0, :1], i, 4)


def calls_with_outputs():
    """(call, the outputs given to it) of each call that writes to tensors of the caller's, the pools aside."""
    bf, i32 = torch.bfloat16, torch.int32
    x, at, f = torch.zeros((2, 2, 64), dtype=bf), torch.zeros(2, dtype=i32), torch.zeros(32, dtype=torch.float64)
    pages = torch.zeros((4, 16, 2, 64), dtype=bf)
    table, lens, starts = torch.zeros((1, 4), dtype=i32), torch.ones(1, dtype=i32), torch.tensor([0, 2], dtype=i32)
    z, q, k, v = torch.zeros((2, 40)), x.clone(), x.clone(), x.clone()
    return [(lambda: gm.keops_rotary(x, at, f, out=x), [x]),
            (lambda: gm.keops_cache_append_rotary(k, k, v, pages, pages.clone(), table, lens, starts, f, out=q), [q]),
            (lambda: gm.keops_cache_read(pages, pages.clone(), table, lens, starts, 2, out=(k, v)), [k, v]),
            (lambda: gm.keops_adjust_logits(z, starts, out=z), [z])]


def check_outputs_and_autograd():
    for call, outs in calls_with_outputs():
        before = [t._version for t in outs]
        call()
        assert [t._version for t in outs] == [n + 1 for n in before]
        # of a tensor that a graph has, the backward pass would not know that it was changed
        outs[0].requires_grad_()
        with pytest.raises(ValueError, match="out must not require a gradient"):
            call()
        with torch.no_grad():
            call()
    y = torch.zeros((2, 2, 64), dtype=torch.bfloat16, requires_grad=True).exp()       # kept for the backward pass
    gm.keops_rotary(y.detach(), torch.zeros(2, dtype=torch.int32), torch.zeros(32, dtype=torch.float64), out=y.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    with torch.inference_mode():
        x = torch.zeros((2, 2, 64), dtype=torch.bfloat16)                             # has no version
    gm.keops_rotary(x, torch.zeros(2, dtype=torch.int32), torch.zeros(32, dtype=torch.float64), out=x)


def test_given_outputs_and_autograd(host):
    check_outputs_and_autograd()


# ---- the compiled way from tensors

@pytest.fixture(scope="module")
def built(tmp_path_factory):
    from torch.utils.cpp_extension import include_paths
    to = tmp_path_factory.mktemp("step_call")
    inc = ["-I", os.path.join(ROOT, "include"), "-isystem", sysconfig.get_paths()["include"]]
    for p in include_paths():
        inc += ["-isystem", p]
    common = ["g++", "-O1", "-shared", "-fPIC", "-std=c++17", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *inc]
    libs = ["-L", os.path.join(os.path.dirname(torch.__file__), "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"]
    for cmd in ([*common, os.path.join(HERE, "step_call_stub.cpp"), "-o", str(to / "libstepstub.so")],
                [*common, "-DPAGED_CALL_DEVICE=c10::DeviceType::CPU", os.path.join(ROOT, "geometric_map_reduce_amd", "native", "step_call.cpp"), "-o",
                 str(to / "_step_call.so"), *libs, "-L", str(to), "-l:libstepstub.so", "-Wl,-rpath,$ORIGIN"]):
        res = subprocess.run(cmd, capture_output=True, text=True)
        assert res.returncode == 0, res.stderr
    return str(to)


def load(folder):
    spec = importlib.util.spec_from_file_location("_step_call", os.path.join(folder, "_step_call.so"))
    short = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(short)
    short.bind(lambda dev: 0)
    return short, ctypes.CDLL(os.path.join(folder, "libstepstub.so"))


def arguments(outputs=False, cache="16"):
    """Plain right arguments of the calls, by name."""
    bf, i32 = torch.bfloat16, torch.int32
    k = torch.zeros((4, 16, 2, 64), dtype=bf)
    ks = vs = None
    if cache == "4":
        k = torch.zeros((4, 16, 2, 32), dtype=torch.uint8).view(torch.float4_e2m1fn_x2)
        ks, vs = (torch.zeros((4, 2, 16, 2), dtype=torch.uint8).view(torch.float8_e8m0fnu) for _ in range(2))
    table, lens, starts = torch.zeros((1, 4), dtype=i32), torch.ones(1, dtype=i32), torch.tensor([0, 1], dtype=i32)
    rows, q = torch.zeros((1, 2, 64), dtype=bf), torch.zeros((1, 4, 64), dtype=bf)
    f, at, one = torch.zeros(16, dtype=torch.float64), torch.zeros(1, dtype=i32), torch.ones(1)
    z = torch.zeros((1, 40))
    held = [k, k.clone(), None, table, lens, ks, vs]
    return dict(
        rotary=[q, at, f, False, 1.0, False, q.clone() if outputs else None],
        append_rotary=[q, rows, rows.clone(), *held, starts, f, at, True, 2, q.clone() if outputs else None],
        read=[*held, starts, 1, 0, None],
        adjust=[z, starts, torch.zeros((1, 9), dtype=i32), lens, lens.clone(), one, one.clone(), one.clone(), torch.zeros((1, 3), dtype=i32),
                torch.zeros((1, 3)), torch.zeros((1, 2), dtype=i32), z.clone() if outputs else None])


@pytest.mark.parametrize("cache", ["16", "4"])
def test_plain_calls_reach_the_library(built, cache):
    short, stub = load(built)
    stub.stub_set(0)
    a = arguments(cache=cache)
    assert short.rotary(*a["rotary"]).shape == (1, 4, 64)
    assert short.append_rotary(*a["append_rotary"]).shape == (1, 4, 64)
    k, v = short.read(*a["read"])
    assert k.shape == v.shape == (1, 2, 64) and k.dtype == torch.bfloat16
    assert short.adjust(*a["adjust"]).shape == (1, 40)
    assert short.adjust(a["adjust"][0], a["adjust"][1], *[None] * 10).shape == (1, 40)
    assert stub.stub_calls() == 5
    a = arguments(outputs=True, cache=cache)
    for name in ("rotary", "append_rotary", "adjust"):
        assert getattr(short, name)(*a[name]) is a[name][-1]


def test_given_outputs_and_autograd_the_short_way(built, host, monkeypatch):
    short, stub = load(built)
    stub.stub_set(0)
    monkeypatch.setattr(step, "_short", short)
    check_outputs_and_autograd()
    assert host == ["keops_cache_read"] * 2 and stub.stub_calls() == 8      # outputs of reading are given the long way


def test_short_way_hands_back_what_it_does_not_take(built):
    """No argument of another kind raises, ends the process or reaches the library."""
    short, stub = load(built)
    stub.stub_set(0)
    for cache in ("16", "4"):
        for name, args in arguments(cache=cache).items():
            call = getattr(short, name)
            for at, x in enumerate(args):
                bads = [object(), "k", [x], torch.zeros((0,)), torch.zeros((3, 3, 3, 3, 3)), torch.zeros((1, 2, 64)).to("meta")]
                for bad in bads:
                    assert call(*args[:at], bad, *args[at + 1:]) is None, (name, at, bad)
            assert call() is None and call(*args, 1) is None
    assert stub.stub_calls() == 0


def every_batched_argument(folder):
    """Each tensor of each call in turn is one that torch.vmap batches: it has no memory of its own."""
    short, stub = load(folder)
    stub.stub_set(0)
    for name, args in arguments(outputs=True).items():
        for at, x in enumerate(args):
            if not isinstance(x, torch.Tensor):
                continue

            def call(t):
                got = getattr(short, name)(*args[:at], t, *args[at + 1:])
                assert got is None, (name, at, got)
                print(name, at, flush=True)
                return t
            torch.vmap(call)(torch.stack([x, x]))
    assert stub.stub_calls() == 0


def test_batched_tensors_are_handed_back(built):
    """In a process of its own: an exception without the interpreter's lock would end it."""
    code = f"import sys; sys.path.insert(0, {HERE!r}); sys.path.insert(0, {ROOT!r}); import test_step_host as t; t.every_batched_argument({built!r})"
    res = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, f"ended with {res.returncode} after\n{res.stdout}\n{res.stderr[-2000:]}"


@pytest.mark.parametrize("outputs", [False, True])
def test_statuses(built, outputs):
    """A refusal is handed back, to be named by the long way; a HIP error is given back as it is, and the call not made again."""
    short, stub = load(built)
    for status in (-1, -2, -3, -4, -5):
        for name, args in arguments(outputs).items():
            stub.stub_set(status)
            got = getattr(short, name)(*args)
            assert stub.stub_calls() == 1
            assert got is None if status != -4 else type(got) is int and got == -4, (name, status, got)


@pytest.mark.parametrize("name,call", [
    ("rotary", lambda a: gm.keops_rotary(*a)), ("append_rotary", lambda a: gm.keops_cache_append_rotary(*a[:5], *a[6:8], a[10], a[11])),
    ("read", lambda a: gm.keops_cache_read(*a[:2], *a[3:5], a[7], 1)), ("adjust", lambda a: gm.keops_adjust_logits(*a))])
def test_a_hip_error_is_raised_once(built, monkeypatch, name, call):
    short, stub = load(built)
    monkeypatch.setattr(step, "_short", short)
    monkeypatch.setattr(binding, "status_string", lambda rc: "HIP error")
    monkeypatch.setattr(step, "_run", lambda *a: pytest.fail("the call went the long way too"))
    stub.stub_set(-4)
    with pytest.raises(gm.KeopsError) as e:
        call(arguments()[name])
    assert e.value.status == -4 and stub.stub_calls() == 1
