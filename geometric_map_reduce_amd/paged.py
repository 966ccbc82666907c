"""Binding of the paged key/value cache and of draft verification (C ABI in
include/keops_mi355x.h, where the operators are defined).

A cache is a pair of page pools ``k_pages``, ``v_pages`` of shape [pages, page_size, heads, dim]
(any order of strides in the first three, the same for both), bfloat16, float16 or float8_e4m3fn with
``k_scale``, ``v_scale`` [heads]; ``weights`` [pages, heads, page_size] float32 holds the
attention that each slot received.  ``page_table`` [sequences, width], ``lens`` [sequences] and
``starts`` [sequences + 1] are int32 tensors on the same device; the calls read none of them on
the host and never synchronise.
"""
from __future__ import annotations

import ctypes
import math

import torch

from .binding import _check, _on_device, _out, _stream, lib

_TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float8_e4m3fn: 2}


class _Cache(ctypes.Structure):
    _fields_ = [("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p), ("weights", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("page_stride", ctypes.c_int64), ("slot_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("pages", ctypes.c_int64), ("page_table", ctypes.c_void_p), ("table_stride", ctypes.c_int64),
                ("lens", ctypes.c_void_p), ("page_size", ctypes.c_int32), ("heads", ctypes.c_int32),
                ("dim", ctypes.c_int32), ("type", ctypes.c_int32), ("table_width", ctypes.c_int32),
                ("seqs", ctypes.c_int32)]


def _vec(t, name, shape, dtype, dev):
    """A dense tensor of this shape (None in it: any size) and type on ``dev``; its address."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype or t.device != dev or t.dim() != len(shape) or not t.is_contiguous() or \
            any(want is not None and want != got for want, got in zip(shape, t.shape)):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape "
                         f"{['any' if s is None else s for s in shape]} on {dev}, got {t.dtype} {list(t.shape)} on {t.device}")
    return t.data_ptr()


def _table(t, name, seqs, dev):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != torch.int32 or t.device != dev or t.dim() != 2 or t.shape[0] != seqs or \
            (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be an int32 tensor [{seqs}, pages of a sequence] on {dev} with contiguous rows")
    return t.data_ptr(), t.stride(0), t.shape[1]


def _cache(k_pages, v_pages, weights, page_table, lens, k_scale, v_scale, scales=True):
    for t, name in ((k_pages, "k_pages"), (v_pages, "v_pages"), (lens, "lens")):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
    dev = k_pages.device
    kind = _TYPES.get(k_pages.dtype)
    if k_pages.dim() != 4 or kind is None or not k_pages.is_cuda or k_pages.stride(3) != 1:
        raise ValueError("k_pages must be a bfloat16, float16 or float8_e4m3fn CUDA tensor "
                         "[pages, page_size, heads, dim] with contiguous rows")
    if v_pages.shape != k_pages.shape or v_pages.dtype != k_pages.dtype or v_pages.device != dev or \
            v_pages.stride() != k_pages.stride():
        raise ValueError("v_pages must have the shape, type, device and strides of k_pages")
    P, ps, H, D = k_pages.shape
    if D not in (64, 96, 128, 256):
        raise ValueError(f"dim must be 64, 96, 128 or 256, got {D}")
    S = lens.shape[0] if lens.dim() == 1 else -1
    c = _Cache()
    c.lens = _vec(lens, "lens", (None,), torch.int32, dev)
    c.page_table, c.table_stride, c.table_width = _table(page_table, "page_table", S, dev)
    c.k_pages, c.v_pages = k_pages.data_ptr(), v_pages.data_ptr()
    # the stride of a dimension of one is never used
    c.page_stride, c.slot_stride, c.head_stride = (st if n > 1 else 0 for st, n in zip(k_pages.stride()[:3], k_pages.shape))
    c.pages, c.page_size, c.heads, c.dim, c.type, c.seqs = P, ps, H, D, kind, S
    if weights is not None:
        c.weights = _vec(weights, "weights", (P, H, ps), torch.float32, dev)
    if kind == 2 and scales:
        if k_scale is None or v_scale is None:
            raise ValueError("a float8_e4m3fn cache needs k_scale and v_scale")
        c.k_scale = _vec(k_scale, "k_scale", (H,), torch.float32, dev)
        c.v_scale = _vec(v_scale, "v_scale", (H,), torch.float32, dev)
    elif k_scale is not None or v_scale is not None:
        raise ValueError("k_scale and v_scale belong to a float8_e4m3fn cache")
    return c, dev


def _rows(t, name, heads, k_pages):
    """Token rows [tokens, heads, dim], 16-bit, heads dense; rows may be part of wider ones."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    D, dtype = k_pages.shape[3], k_pages.dtype
    if t.dim() != 3 or t.dtype not in (torch.bfloat16, torch.float16) or t.device != k_pages.device or t.shape[2] != D or \
            (heads is not None and t.shape[1] != heads) or (dtype.itemsize == 2 and t.dtype != dtype):
        raise ValueError(f"{name} must be [tokens, {'heads' if heads is None else heads}, {D}], of the cache's type "
                         f"(bfloat16 or float16 with an 8-bit cache), on {k_pages.device}")
    if t.numel() and (t.stride(2) != 1 or (t.shape[1] > 1 and t.stride(1) != D)):
        raise ValueError(f"{name} must have dense [heads, dim] rows")
    if t.data_ptr() % 16 or (t.shape[0] > 1 and t.stride(0) % 8):
        raise ValueError(f"{name} must be 16-byte aligned, its rows a multiple of 16 bytes apart")
    return t.data_ptr(), t.stride(0) if t.shape[0] > 1 else t.shape[1] * D


def _keep(stream, dev, *tensors):
    """Tensors made here for a call on another stream than the current one belong to that stream too."""
    if stream is None:
        return
    s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream), device=dev)
    if s.cuda_stream != torch.cuda.current_stream(dev).cuda_stream:
        for t in tensors:
            if t is not None:
                t.record_stream(s)


def _graph_workspace(name, dev, *args):
    """(address, bytes, tensor) of a call's workspace under stream capture, from the graph's own pool, where it
    lives as long as the graph; nothing otherwise: the library has its own."""
    if not torch.cuda.is_current_stream_capturing():
        return None, 0, None
    need = ctypes.c_int64(0)
    _check(name, getattr(lib(), name + "_workspace")(*args, ctypes.byref(need)))
    if need.value == 0:
        return None, 0, None
    buf = torch.empty(need.value + 256, dtype=torch.uint8, device=dev)
    return (buf.data_ptr() + 255) // 256 * 256, need.value, buf


def keops_cache_append(k, v, k_pages, v_pages, page_table, lens, starts, weights=None, k_scale=None, v_scale=None,
                       stream=None):
    """Write rows starts[s] .. starts[s+1] of k and v [tokens, heads, dim] to the last slots of sequence s
    (``lens`` counts them already); clear those slots' ``weights``."""
    c, dev = _cache(k_pages, v_pages, weights, page_table, lens, k_scale, v_scale)
    kp, ks = _rows(k, "k", c.heads, k_pages)
    vp, vs = _rows(v, "v", c.heads, k_pages)
    if v.shape != k.shape or v.dtype != k.dtype:
        raise ValueError("v must have the shape and type of k")
    st = _vec(starts, "starts", (c.seqs + 1,), torch.int32, dev)
    with _on_device(dev):
        rc = lib().keops_cache_append(ctypes.addressof(c), kp, vp, ks, vs, _TYPES[k.dtype], st, k.shape[0], _stream(stream, dev))
    _check("keops_cache_append", rc)


def keops_paged_attention(q, k_pages, v_pages, page_table, lens, starts, max_q, max_len, scale=None, window=0, weights=None,
                          decay=0.0, k_scale=None, v_scale=None, out=None, lse=None, stream=None):
    """Causal attention of the new tokens' queries q [tokens, query heads, dim] over the cache: (out, lse).

    ``max_q`` and ``max_len`` bound the new tokens and the slots of any sequence; ``scale`` is
    1 / sqrt(dim) unless given; ``window`` > 0 limits a token to that many slots, its own included.
    With ``weights``, every slot's becomes decay * old + the attention it received in this call."""
    c, dev = _cache(k_pages, v_pages, weights, page_table, lens, k_scale, v_scale)
    qp, qs = _rows(q, "q", None, k_pages)
    T, heads, D = q.shape
    if heads < 1 or heads % c.heads:
        raise ValueError(f"the query heads must be a multiple of the cache's {c.heads}, got {heads}")
    st = _vec(starts, "starts", (c.seqs + 1,), torch.int32, dev)
    max_q, max_len, window = int(max_q), int(max_len), int(window)
    if min(max_q, max_len, window) < 0 or max(max_q, max_len, window) > 2**31 - 1:
        raise ValueError("max_q, max_len and window must be in [0, 2^31)")
    given_out, given_lse = out, lse
    out = _out(out, (T, heads, D), dev, q.dtype)
    lse = _out(lse, (T, heads), dev, name="lse")
    s = _stream(stream, dev)
    kind = _TYPES[q.dtype]
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    with _on_device(dev):
        ws, nbytes, buf = _graph_workspace("keops_paged_attention", dev, ctypes.addressof(c), kind, heads, T, max_q, max_len,
                                           window)
        rc = lib().keops_paged_attention(ctypes.addressof(c), qp, qs, kind, heads, st, T, max_q, max_len, scale, window,
                                         float(decay), out.data_ptr(), lse.data_ptr(), ws, nbytes, s)
    _check("keops_paged_attention", rc)
    _keep(stream, dev, None if given_out is not None else out, None if given_lse is not None else lse, buf)
    return out, lse


def keops_cache_evict(k_pages, v_pages, weights, page_table, lens, new_table, budget, sink=0, recent=0, kept=None,
                      new_lens=None, stream=None):
    """Keep ``budget`` slots of every sequence and head: the first ``sink``, the last ``recent``, and those with
    the largest weights; move them to the pages of ``new_table``.  Returns (kept [sequences, heads, budget]
    old slot numbers or -1, new lens).  The scales of an 8-bit cache are not needed."""
    c, dev = _cache(k_pages, v_pages, weights, page_table, lens, None, None, scales=False)
    if weights is None:
        raise ValueError("eviction needs weights")
    nt, nstride, nwidth = _table(new_table, "new_table", c.seqs, dev)
    budget, sink, recent = int(budget), int(sink), int(recent)
    if budget < 1 or sink < 0 or recent < 0 or sink + recent > budget:
        raise ValueError("need budget >= 1, sink >= 0, recent >= 0 and sink + recent <= budget")
    if nwidth < min(-(-budget // c.page_size), c.table_width):
        raise ValueError("new_table has too few pages for the budget")
    given_kept, given_lens = kept, new_lens
    kept = _out(kept, (c.seqs, c.heads, budget), dev, torch.int32, name="kept")
    new_lens = _out(new_lens, (c.seqs,), dev, torch.int32, name="new_lens")
    with _on_device(dev):
        rc = lib().keops_cache_evict(ctypes.addressof(c), nt, nstride, nwidth, budget, sink, recent, kept.data_ptr(),
                                     new_lens.data_ptr(), _stream(stream, dev))
    _check("keops_cache_evict", rc)
    _keep(stream, dev, None if given_kept is not None else kept, None if given_lens is not None else new_lens)
    return kept, new_lens


def keops_verify_draft(target, draft, tokens, counts, u_accept, u_sample, out=None, accepted=None, stream=None):
    """Drafted ``tokens`` [sequences, drafts] (the first counts[s] of them) against the target's probabilities
    [sequences, drafts + 1, vocab] and the draft's [sequences, drafts, vocab] (None: certain), with given uniform
    numbers.  Returns (tokens [sequences, drafts + 1]: taken, then the new one, then -1; accepted [sequences])."""
    if not isinstance(target, torch.Tensor) or not isinstance(tokens, torch.Tensor):
        raise TypeError("target and tokens must be torch.Tensors")
    if target.dim() != 3 or not target.is_cuda or tokens.dim() != 2:
        raise ValueError("target must be a CUDA tensor [sequences, drafts + 1, vocab], tokens [sequences, drafts]")
    dev, (S, K), V = target.device, tokens.shape, target.shape[2]
    if V < 1:
        raise ValueError("the vocabulary is empty")
    f32, i32 = torch.float32, torch.int32
    args = [_vec(target, "target", (S, K + 1, V), f32, dev),
            None if draft is None else _vec(draft, "draft", (S, K, V), f32, dev),
            _vec(tokens, "tokens", (S, K), i32, dev), _vec(counts, "counts", (S,), i32, dev),
            _vec(u_accept, "u_accept", (S, K), f32, dev), _vec(u_sample, "u_sample", (S,), f32, dev)]
    if K == 0 and draft is not None:
        args[1] = None
    given_out, given_acc = out, accepted
    out = _out(out, (S, K + 1), dev, i32)
    accepted = _out(accepted, (S,), dev, i32, name="accepted")
    with _on_device(dev):
        ws, nbytes, buf = _graph_workspace("keops_verify_draft", dev, S, K, V)
        rc = lib().keops_verify_draft(*args, S, K, V, out.data_ptr(), accepted.data_ptr(), ws, nbytes, _stream(stream, dev))
    _check("keops_verify_draft", rc)
    _keep(stream, dev, None if given_out is not None else out, None if given_acc is not None else accepted, buf)
    return out, accepted
