"""Binding of the paged key/value cache and of draft verification (C ABI in
include/keops_mi355x.h, where the operators are defined).

A cache is a pair of page pools ``k_pages``, ``v_pages`` of shape [pages, page_size, heads, dim]
(any order of strides in the first three, the same for both), bfloat16, float16, float8_e4m3fn with
``k_scale``, ``v_scale`` [heads], or float4_e2m1fn_x2 (two values an element: [.., dim / 2]) with ``k_scale``,
``v_scale`` [pages, heads, page_size, dim / 32] float8_e8m0fnu, a power of two for 32 columns;
``weights`` [pages, heads, page_size] float32 holds the
attention that each slot received.  ``page_table`` [sequences, width], ``lens`` [sequences] and
``starts`` [sequences + 1] are int32 tensors on the same device; the calls read none of them on
the host and never synchronise.

None of these has a gradient: outputs are constants to autograd, also where an input requires one,
and writes to the pools and to ``weights`` do not raise the tensors' version counters.

Each call first goes the short way (native/paged_call.cpp), which takes plain arguments on the
current stream in a microsecond or two and hands back, undone, whatever is anything else; that is
taken, or refused by name, here.  A HIP error is raised as it comes: some of a call's launches may
have been made by then, so the call is not made again.
"""
from __future__ import annotations

import ctypes
import importlib
import math
import os
import struct

import torch

from .binding import LIB_PATH, _check, _out, _raw_stream, _stream, lib

_TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float8_e4m3fn: 2, torch.float4_e2m1fn_x2: 4}


# keops_cache_t: k_pages, v_pages, weights, k_scale, v_scale; page, slot and head stride, pages;
# page_table, table_stride, lens; page_size, heads, dim, type, table_width, seqs
_CACHE = struct.Struct("=5Q4qQqQ6i")


def _tensor(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    return t


def _vec(t, name, shape, dtype, dev):
    """The address of a dense tensor of this shape and type on device number ``dev``."""
    try:
        if t.dtype is dtype and t.get_device() == dev and t.shape == shape and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        _tensor(t, name)
        raise
    raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {list(shape)} on cuda:{dev}, "
                     f"got {t.dtype} {list(t.shape)} on {t.device}")


def _table(t, name, seqs, dev):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    shape, strides = t.shape, t.stride()
    if len(shape) != 2 or shape[0] != seqs or t.dtype is not torch.int32 or t.get_device() != dev or \
            (strides[1] != 1 and shape[1] > 1):
        raise ValueError(f"{name} must be an int32 tensor [{seqs}, pages of a sequence] on cuda:{dev} with contiguous rows")
    return t.data_ptr(), strides[0], shape[1]


def _cache(k_pages, v_pages, weights, page_table, lens, k_scale, v_scale, scales=True):
    """(the structure of the C ABI, the device's number, sequences, (heads, dim, type), page size, pages of a sequence)."""
    if not (isinstance(k_pages, torch.Tensor) and isinstance(v_pages, torch.Tensor) and isinstance(lens, torch.Tensor)):
        _tensor(k_pages, "k_pages"), _tensor(v_pages, "v_pages"), _tensor(lens, "lens")
    dev, dtype, shape, strides = k_pages.get_device(), k_pages.dtype, k_pages.shape, k_pages.stride()
    kind = _TYPES.get(dtype)
    if len(shape) != 4 or kind is None or dev < 0 or strides[3] != 1:
        raise ValueError("k_pages must be a bfloat16, float16, float8_e4m3fn or float4_e2m1fn_x2 CUDA tensor "
                         "[pages, page_size, heads, dim] with contiguous rows")
    if v_pages.shape != shape or v_pages.dtype is not dtype or v_pages.get_device() != dev or v_pages.stride() != strides:
        raise ValueError("v_pages must have the shape, type, device and strides of k_pages")
    P, ps, H, D = shape
    two = 1
    if kind == 4:       # an element of two values
        D, two = 2 * D, 2
    if D not in (64, 96, 128, 256):
        raise ValueError(f"dim must be 64, 96, 128 or 256, got {D}")
    if lens.dim() != 1 or lens.dtype is not torch.int32 or lens.get_device() != dev or not lens.is_contiguous():
        raise ValueError(f"lens must be a contiguous int32 tensor [sequences] on cuda:{dev}")
    S = lens.shape[0]
    table, table_stride, width = _table(page_table, "page_table", S, dev)
    w = ks = vs = 0
    if weights is not None:
        w = _vec(weights, "weights", (P, H, ps), torch.float32, dev)
    if kind == 2:
        if scales:
            if k_scale is None or v_scale is None:
                raise ValueError("a float8_e4m3fn cache needs k_scale and v_scale")
            ks = _vec(k_scale, "k_scale", (H,), torch.float32, dev)
            vs = _vec(v_scale, "v_scale", (H,), torch.float32, dev)
    elif kind == 4:
        if k_scale is None or v_scale is None:
            raise ValueError("a float4_e2m1fn_x2 cache needs k_scale and v_scale")
        ks = _vec(k_scale, "k_scale", (P, H, ps, D // 32), torch.float8_e8m0fnu, dev)
        vs = _vec(v_scale, "v_scale", (P, H, ps, D // 32), torch.float8_e8m0fnu, dev)
    elif k_scale is not None or v_scale is not None:
        raise ValueError("k_scale and v_scale belong to a float8_e4m3fn or float4_e2m1fn_x2 cache")
    # the stride of a dimension of one is never used
    c = _CACHE.pack(k_pages.data_ptr(), v_pages.data_ptr(), w, ks, vs, strides[0] * two if P > 1 else 0,
                    strides[1] * two if ps > 1 else 0, strides[2] * two if H > 1 else 0, P, table, table_stride, lens.data_ptr(), ps, H, D, kind,
                    width, S)
    return c, dev, S, (H, D, dtype), ps, width


_short = None


def _module(name):
    """A module of the short way; nothing before the library is built, which the long way reports."""
    if not os.path.exists(LIB_PATH):
        return None
    lib()
    try:
        module = importlib.import_module("." + name, __package__)
    except ImportError as e:
        raise RuntimeError(f"the module {name} is missing or broken: build it first "
                           "(python -m geometric_map_reduce_amd.build)") from e
    module.bind(_raw_stream)
    return module


def _native():
    global _short
    _short = _module("_paged_call")
    return _short


def _ended(name, got):
    """What the short way gave; raises on a status."""
    if type(got) is int:
        _check(name, got)
    return got


_HALF = (torch.bfloat16, torch.float16)


def _rows(t, name, heads, cache, dev):
    """Token rows [tokens, heads, dim], 16-bit, heads dense; rows may be part of wider ones."""
    _tensor(t, name)
    H, D, held = cache
    shape, dtype = t.shape, t.dtype
    if len(shape) != 3 or dtype not in _HALF or t.get_device() != dev or shape[2] != D or \
            (heads is not None and shape[1] != heads) or (held in _HALF and dtype is not held):
        raise ValueError(f"{name} must be [tokens, {'heads' if heads is None else heads}, {D}], of the cache's type "
                         f"(bfloat16 or float16 with an 8-bit or 4-bit cache), on cuda:{dev}")
    T, h, _ = shape
    s0, s1, s2 = t.stride()
    if T and (s2 != 1 or (h > 1 and s1 != D)):
        raise ValueError(f"{name} must have dense [heads, dim] rows")
    at = t.data_ptr()
    if at % 16 or (T > 1 and s0 % 8):
        raise ValueError(f"{name} must be 16-byte aligned, its rows a multiple of 16 bytes apart")
    return at, s0 if T > 1 else h * D


def _run(name, dev, stream, fn, *args):
    """fn(*args, stream) with device ``dev`` current; raises on a status."""
    if torch.cuda.current_device() != dev:
        with torch.cuda.device(dev):
            return _run(name, dev, stream, fn, *args)
    rc = fn(*args, _stream(stream, torch.device("cuda", dev)) if stream is not None or _raw_stream is None else _raw_stream(dev))
    if rc:
        _check(name, rc)


def _other(stream, dev):
    """The stream that a call names, where it is not the current one; else None.

    What the call makes comes from that stream's memory: a block of the current stream's may still be in use by
    work queued there, of which the other stream knows nothing."""
    if stream is None:
        return None
    given = isinstance(stream, torch.cuda.Stream)
    handle = stream.cuda_stream if given else int(stream)
    if handle == torch.cuda.current_stream(dev).cuda_stream:
        return None
    if given:
        return stream
    # ExternalStream takes the default stream's handle, 0, for none
    return torch.cuda.ExternalStream(handle, device=dev) if handle else torch.cuda.default_stream(dev)


def _keep(other, dev, *tensors):
    """Outputs made on another stream than the current one, where the caller reads them, belong to that too."""
    if other is not None:
        for t in tensors:
            if t is not None:
                t.record_stream(torch.cuda.current_stream(dev))


def _graph_workspace(name, dev, *args):
    """(address, bytes, tensor) of a call's workspace where the current stream is captured, from the graph's own
    pool, where it lives as long as the graph; nothing otherwise: the library has its own."""
    if not torch.cuda.is_current_stream_capturing():
        return None, 0, None
    need = ctypes.c_int64(0)
    with torch.cuda.device(dev):
        _check(name, getattr(lib(), name + "_workspace")(*args, ctypes.byref(need)))
    if need.value == 0:
        return None, 0, None
    buf = torch.empty(need.value + 256, dtype=torch.uint8, device=dev)
    return (buf.data_ptr() + 255) // 256 * 256, need.value, buf


def keops_cache_append(k, v, k_pages, v_pages, page_table, lens, starts, weights=None, k_scale=None, v_scale=None,
                       stream=None):
    """Write rows starts[s] .. starts[s+1] of k and v [tokens, heads, dim] to the last slots of sequence s
    (``lens`` counts them already); clear those slots' ``weights``.  No gradient."""
    if stream is None:
        short = _short or _native()
        got = short and short.append(k, v, k_pages, v_pages, weights, page_table, lens, k_scale, v_scale, starts)
        if got:
            _ended("keops_cache_append", got)
            return
    c, dev, S, cache, _, _ = _cache(k_pages, v_pages, weights, page_table, lens, k_scale, v_scale)
    kp, ks = _rows(k, "k", cache[0], cache, dev)
    vp, vs = _rows(v, "v", cache[0], cache, dev)
    if v.shape != k.shape or v.dtype is not k.dtype:
        raise ValueError("v must have the shape and type of k")
    st = _vec(starts, "starts", (S + 1,), torch.int32, dev)
    _run("keops_cache_append", dev, stream, lib().keops_cache_append, c, kp, vp, ks, vs, _TYPES[k.dtype], st,
         k.shape[0])


def keops_paged_attention(q, k_pages, v_pages, page_table, lens, starts, max_q, max_len, scale=None, window=0, weights=None,
                          decay=0.0, k_scale=None, v_scale=None, out=None, lse=None, stream=None):
    """Causal attention of the new tokens' queries q [tokens, query heads, dim] over the cache: (out, lse).

    ``max_q`` and ``max_len`` bound the new tokens and the slots of any sequence; ``scale`` is
    1 / sqrt(dim) unless given; ``window`` > 0 limits a token to that many slots, its own included.
    With ``weights``, every slot's becomes decay * old + the attention it received in this call, from all of
    q's rows: drafted tokens that are refused later have had their part.  No gradient."""
    if stream is None:
        short = _short or _native()
        got = short and short.attention(q, k_pages, v_pages, weights, page_table, lens, k_scale, v_scale, starts, max_q, max_len,
                                        scale, window, decay, out, lse)
        if got:
            return _ended("keops_paged_attention", got)
    c, dev, S, cache, _, _ = _cache(k_pages, v_pages, weights, page_table, lens, k_scale, v_scale)
    qp, qs = _rows(q, "q", None, cache, dev)
    T, heads, D = q.shape
    if heads < 1 or heads % cache[0]:
        raise ValueError(f"the query heads must be a multiple of the cache's {cache[0]}, got {heads}")
    st = _vec(starts, "starts", (S + 1,), torch.int32, dev)
    max_q, max_len, window = int(max_q), int(max_len), int(window)
    if min(max_q, max_len, window) < 0 or max(max_q, max_len, window) > 2**31 - 1:
        raise ValueError("max_q, max_len and window must be in [0, 2^31)")
    kind = _TYPES[q.dtype]
    other = _other(stream, dev)
    with torch.cuda.stream(other):
        made = (None if out is not None else torch.empty_like(q) if q.is_contiguous() else q.new_empty((T, heads, D)),
                None if lse is not None else q.new_empty((T, heads), dtype=torch.float32))
        out = made[0] if out is None else _out(out, (T, heads, D), q.device, q.dtype)
        lse = made[1] if lse is None else _out(lse, (T, heads), q.device, name="lse")
        ws, nbytes, buf = _graph_workspace("keops_paged_attention", dev, c, kind, heads, T, max_q, max_len, window)
    _run("keops_paged_attention", dev, stream, lib().keops_paged_attention, c, qp, qs, kind, heads, st, T, max_q, max_len,
         1.0 / math.sqrt(D) if scale is None else float(scale), window, float(decay), out.data_ptr(), lse.data_ptr(), ws, nbytes)
    _keep(other, dev, *made)
    return out, lse


def keops_cache_evict(k_pages, v_pages, weights, page_table, lens, new_table, budget, sink=0, recent=0, kept=None,
                      new_lens=None, stream=None, k_scale=None, v_scale=None):
    """Keep ``budget`` slots of every sequence and head: the first ``sink``, the last ``recent``, and those with
    the largest weights; move them to the pages of ``new_table``.  Returns (kept [sequences, heads, budget]
    old slot numbers or -1, new lens).  Slots whose page the table lacks are left out, and not counted in the
    new lens.  The scales of an 8-bit cache are not needed; those of a 4-bit cache belong to its slots and move
    with them."""
    if stream is None:
        short = _short or _native()
        got = short and short.evict(k_pages, v_pages, weights, page_table, lens, k_scale, v_scale, new_table, budget, sink, recent, kept,
                                    new_lens)
        if got:
            return _ended("keops_cache_evict", got)
    c, dev, S, (H, _, _), ps, width = _cache(k_pages, v_pages, weights, page_table, lens, k_scale, v_scale, scales=False)
    if weights is None:
        raise ValueError("eviction needs weights")
    nt, nstride, nwidth = _table(new_table, "new_table", S, dev)
    budget, sink, recent = int(budget), int(sink), int(recent)
    if not 1 <= budget < 2**31 or sink < 0 or recent < 0 or sink + recent > budget:
        raise ValueError("need 1 <= budget < 2^31, sink >= 0, recent >= 0 and sink + recent <= budget")
    if nwidth < min(-(-budget // ps), width):
        raise ValueError("new_table has too few pages for the budget")
    other = _other(stream, dev)
    with torch.cuda.stream(other):
        made = (None if kept is not None else torch.empty((S, H, budget), dtype=torch.int32, device=k_pages.device),
                None if new_lens is not None else torch.empty((S,), dtype=torch.int32, device=k_pages.device))
    kept = made[0] if kept is None else _out(kept, (S, H, budget), k_pages.device, torch.int32, name="kept")
    new_lens = made[1] if new_lens is None else _out(new_lens, (S,), k_pages.device, torch.int32, name="new_lens")
    _run("keops_cache_evict", dev, stream, lib().keops_cache_evict, c, nt, nstride, nwidth, budget, sink, recent,
         kept.data_ptr(), new_lens.data_ptr())
    _keep(other, dev, *made)
    return kept, new_lens


def keops_verify_draft(target, draft, tokens, counts, u_accept, u_sample, out=None, accepted=None, stream=None):
    """Drafted ``tokens`` [sequences, drafts] (the first counts[s] of them) against the target's probabilities
    [sequences, drafts + 1, vocab] and the draft's [sequences, drafts, vocab] (None: certain), with given uniform
    numbers.  Returns (tokens [sequences, drafts + 1]: taken, then the new one, then -1; accepted [sequences])."""
    if stream is None:
        short = _short or _native()
        got = short and short.verify(target, draft, tokens, counts, u_accept, u_sample, out, accepted)
        if got:
            return _ended("keops_verify_draft", got)
    _tensor(target, "target"), _tensor(tokens, "tokens")
    dev = target.get_device()
    if target.dim() != 3 or dev < 0 or tokens.dim() != 2:
        raise ValueError("target must be a CUDA tensor [sequences, drafts + 1, vocab], tokens [sequences, drafts]")
    (S, K), V = tokens.shape, target.shape[2]
    if V < 1:
        raise ValueError("the vocabulary is empty")
    f32, i32 = torch.float32, torch.int32
    tp = _vec(target, "target", (S, K + 1, V), f32, dev)
    dp = None if draft is None else _vec(draft, "draft", (S, K, V), f32, dev)
    xp, cp = _vec(tokens, "tokens", (S, K), i32, dev), _vec(counts, "counts", (S,), i32, dev)
    ap, sp = _vec(u_accept, "u_accept", (S, K), f32, dev), _vec(u_sample, "u_sample", (S,), f32, dev)
    other = _other(stream, dev)
    with torch.cuda.stream(other):
        made = (None if out is not None else torch.empty((S, K + 1), dtype=i32, device=target.device),
                None if accepted is not None else torch.empty((S,), dtype=i32, device=target.device))
        out = made[0] if out is None else _out(out, (S, K + 1), target.device, i32)
        accepted = made[1] if accepted is None else _out(accepted, (S,), target.device, i32, name="accepted")
        ws, nbytes, buf = _graph_workspace("keops_verify_draft", dev, S, K, V)
    _run("keops_verify_draft", dev, stream, lib().keops_verify_draft, tp, dp if K else None, xp, cp, ap, sp, S, K, V, out.data_ptr(),
         accepted.data_ptr(), ws, nbytes)
    _keep(other, dev, *made)
    return out, accepted
