"""Binding of the operators around the paged key/value cache: rotary positions, the append that rotates, reading
slots back, and the adjustment of logits (C ABI in include/keops_mi355x.h, where they are defined).

Conventions are those of ``paged.py``.  ``keops_rotary`` is differentiated by calling it on the gradient with
``inverse=True``; to autograd the outputs of all of these are constants.  A tensor given as ``out`` has its version
counter raised, and is refused where it requires a gradient and gradients are enabled.

Each call first goes the short way (native/step_call.cpp), as the paged calls do.
"""
from __future__ import annotations

import math
import struct

import torch

from .binding import lib
from .paged import (_HALF, _TYPES, _cache, _ended, _keep, _module, _other, _rows, _run, _table, _tensor, _vec)

_ROWS = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 3}

# keops_rotary_t: freqs; factor; pairs, interleaved
_ROTARY = struct.Struct("=Qd2i")
# keops_logit_rules_t: starts, text; text_stride; lens, prompt_lens, repetition, presence, frequency, bias_tokens, bias,
# mask; mask_stride; seqs, text_width, biases
_RULES = struct.Struct("=2Qq8Qq3i4x")

_short = None


def _native():
    global _short
    _short = _module("_step_call")
    return _short


def keops_rotary_frequencies(dim, base=10000.0, scaling=None, factor=1.0, length=None, slow=1.0, fast=4.0, device=None):
    """The frequencies of ``dim`` rotated columns, base^(-2 i / dim) for pair i, as float64 [dim / 2].

    ``scaling`` lets a model read texts ``factor`` times as long as it was trained on:
    "linear" divides all by the factor; "base" raises the base so that the slowest pair is divided by the factor and
    the fastest stays; "parts" goes by the turns that a pair makes within the ``length`` tokens of the training:
    more than ``fast`` and it stays, fewer than ``slow`` and it is divided, in between some of both, linear in the turns."""
    dim, base, factor = int(dim), float(base), float(factor)
    if dim < 2 or dim % 2 or not base > 0 or not factor > 0:
        raise ValueError("need an even dim >= 2, base > 0 and factor > 0")
    if scaling == "base":
        if dim < 4:
            raise ValueError("scaling the base needs two pairs")
        base *= factor ** (dim / (dim - 2))
    i = torch.arange(dim // 2, dtype=torch.float64)
    freqs = torch.exp(-(2 * i / dim) * math.log(base))
    if scaling == "linear":
        freqs = freqs / factor
    elif scaling == "parts":
        if length is None or not 0 <= slow < fast:
            raise ValueError("scaling by parts needs the length of the training's texts, and 0 <= slow < fast")
        share = ((length * freqs / (2 * math.pi) - slow) / (fast - slow)).clamp(0, 1)
        freqs = share * freqs + (1 - share) * freqs / factor
    elif scaling not in (None, "base"):
        raise ValueError(f"scaling must be None, 'linear', 'base' or 'parts', got {scaling!r}")
    return freqs.to(device)


def _rotary(freqs, interleaved, factor, dim, dev):
    _tensor(freqs, "freqs")
    if freqs.dim() != 1 or 2 * freqs.shape[0] > dim:
        raise ValueError(f"freqs must have one dimension, of at most {dim // 2}")
    factor = float(factor)
    if not math.isfinite(factor):
        raise ValueError("factor must be finite")
    return _ROTARY.pack(_vec(freqs, "freqs", (freqs.shape[0],), torch.float64, dev), factor, freqs.shape[0], bool(interleaved))


def _dense_heads(t, name):
    """The distance of token rows [tokens, heads, dim] with dense heads."""
    T, H, D = t.shape
    s0, s1, s2 = t.stride()
    if t.numel() and ((D > 1 and s2 != 1) or (H > 1 and s1 != D)):
        raise ValueError(f"{name} must have dense [heads, dim] rows")
    return s0 if T > 1 else H * D


def _given(t, name, like, shape):
    _tensor(t, name)
    if t.dtype is not like.dtype or t.device != like.device or t.shape != torch.Size(shape):
        raise ValueError(f"{name} must be a {like.dtype} tensor of shape {list(shape)} on {like.device}")
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{name} must not require a gradient: the call has none")
    return t


def _written(*tensors):
    """Tells autograd that the caller's tensors have changed."""
    for t in tensors:
        if not t.is_inference():
            torch.autograd.graph.increment_version(t)


def keops_rotary(x, positions, freqs, interleaved=False, factor=1.0, inverse=False, out=None, stream=None):
    """x [tokens, heads, dim] with the first 2 len(freqs) columns of each head turned by positions[t] * freqs[i]:
    columns i and i + len(freqs), or, ``interleaved``, 2 i and 2 i + 1.  ``factor`` multiplies what turns.
    bfloat16, float16 or float32; ``positions`` int32 [tokens], ``freqs`` float64.

    ``inverse`` turns the other way: of the gradient with respect to the output it makes the one with respect to x.
    No gradient of its own: the output is a constant to autograd, also where x requires one.  ``out`` may be x."""
    if stream is None:
        short = _short or _native()
        got = short and short.rotary(x, positions, freqs, interleaved, factor, inverse, out)
        if got is not None and got is not False:
            return _ended("keops_rotary", got)
    _tensor(x, "x"), _tensor(positions, "positions")
    dev, kind = x.get_device(), _ROWS.get(x.dtype)
    if x.dim() != 3 or kind is None or dev < 0:
        raise ValueError("x must be a bfloat16, float16 or float32 CUDA tensor [tokens, heads, dim]")
    T, H, D = x.shape
    if D < 1:
        raise ValueError("dim must be at least 1")
    r = _rotary(freqs, interleaved, factor, D, dev)
    at = _vec(positions, "positions", (T,), torch.int32, dev)
    xs = _dense_heads(x, "x")
    other = _other(stream, dev)
    with torch.cuda.stream(other):
        made = x.new_empty((T, H, D)) if out is None else None
    out = made if out is None else _given(out, "out", x, (T, H, D))
    _run("keops_rotary", dev, stream, lib().keops_rotary, x.data_ptr(), xs, kind, T, H, D, at, r, bool(inverse), out.data_ptr(),
         _dense_heads(out, "out"))
    _keep(other, dev, made)
    if made is None:
        _written(out)
    return out


def keops_cache_append_rotary(q, k, v, k_pages, v_pages, page_table, lens, starts, freqs, positions=None, interleaved=False,
                              factor=1.0, weights=None, k_scale=None, v_scale=None, out=None, stream=None):
    """``keops_cache_append`` of k, rotated, and v, and the rotated queries q [tokens, query heads, dim], which are
    returned (``out``: where to, not into q).  A token's position is that of ``positions`` int32 [tokens], or its slot's number.
    Rotation as in ``keops_rotary``; an 8-bit or 4-bit cache holds what is nearest to the rotated key itself.  Rows of
    tokens in no sequence are not written.  No gradient."""
    if stream is None:
        short = _short or _native()
        got = short and short.append_rotary(q, k, v, k_pages, v_pages, weights, page_table, lens, k_scale, v_scale, starts, freqs,
                                            positions, interleaved, factor, out)
        if got is not None and got is not False:
            return _ended("keops_cache_append_rotary", got)
    c, dev, S, cache, _, _ = _cache(k_pages, v_pages, weights, page_table, lens, k_scale, v_scale)
    qp, qs = _rows(q, "q", None, cache, dev)
    kp, ks = _rows(k, "k", cache[0], cache, dev)
    vp, vs = _rows(v, "v", cache[0], cache, dev)
    if v.shape != k.shape or v.dtype is not k.dtype:
        raise ValueError("v must have the shape and type of k")
    if q.shape[0] != k.shape[0] or q.dtype is not k.dtype:
        raise ValueError("q must have the tokens and the type of k")
    T, heads, D = q.shape
    st = _vec(starts, "starts", (S + 1,), torch.int32, dev)
    at = 0 if positions is None else _vec(positions, "positions", (T,), torch.int32, dev)
    r = _rotary(freqs, interleaved, factor, D, dev)
    other = _other(stream, dev)
    with torch.cuda.stream(other):
        made = q.new_empty((T, heads, D)) if out is None else None
    out = made if out is None else _given(out, "out", q, (T, heads, D))
    _run("keops_cache_append_rotary", dev, stream, lib().keops_cache_append_rotary, c, qp, kp, vp, qs, ks, vs, _TYPES[k.dtype], heads,
         st, T, at, r, out.data_ptr(), _dense_heads(out, "out"))
    _keep(other, dev, made)
    if made is None:
        _written(out)
    return out


def keops_cache_read(k_pages, v_pages, page_table, lens, starts, tokens, dtype=None, k_scale=None, v_scale=None, out=None, stream=None):
    """The keys and values in the slots of every sequence's last starts[s+1] - starts[s] tokens, ``tokens`` of them in
    all, as 16-bit rows (k, v) [tokens, heads, dim]: whole sequences where starts adds up the lens.  ``dtype``: bfloat16
    (unless given) or float16 of an 8-bit or 4-bit cache, else the cache's own.  ``out``: a pair of tensors to write to.
    Rows of absent slots are 0; rows of tokens in no sequence are not written.  No gradient."""
    if dtype is None:
        dtype = k_pages.dtype if isinstance(k_pages, torch.Tensor) and k_pages.dtype in _HALF else torch.bfloat16
    if stream is None and out is None:
        short = _short or _native()
        got = short and short.read(k_pages, v_pages, None, page_table, lens, k_scale, v_scale, starts, tokens, _TYPES.get(dtype), None)
        if got is not None and got is not False:
            return _ended("keops_cache_read", got)
    c, dev, S, (H, D, held), _, _ = _cache(k_pages, v_pages, None, page_table, lens, k_scale, v_scale)
    if dtype not in _HALF or (held in _HALF and dtype is not held):
        raise ValueError("dtype must be the cache's type (bfloat16 or float16 of an 8-bit or 4-bit cache)")
    T = int(tokens)
    if not 0 <= T < 2**31:
        raise ValueError("tokens must be in [0, 2^31)")
    st = _vec(starts, "starts", (S + 1,), torch.int32, dev)
    other = _other(stream, dev)
    with torch.cuda.stream(other):
        made = tuple(torch.empty((T, H, D), dtype=dtype, device=k_pages.device) if out is None else None for _ in range(2))
    k, v = made if out is None else (_given(t, "out", torch.empty(0, dtype=dtype, device=k_pages.device), (T, H, D)) for t in out)
    _run("keops_cache_read", dev, stream, lib().keops_cache_read, c, k.data_ptr(), v.data_ptr(), _dense_heads(k, "out"),
         _dense_heads(v, "out"), _TYPES[dtype], st, T)
    _keep(other, dev, *made)
    if out is not None:
        _written(k, v)
    return k, v


def keops_adjust_logits(logits, starts, tokens=None, lens=None, prompt_lens=None, repetition=None, presence=None, frequency=None,
                        bias_tokens=None, bias=None, mask=None, out=None, stream=None):
    """``logits`` [rows, vocab] (bfloat16, float16 or float32) by penalties, biases and masks, in this order.

    Rows starts[s] .. starts[s+1] are those of sequence s, whose text ``tokens`` int32 [sequences, width] has lens[s]
    tokens, the rows' own last: a row goes by the text up to its own token, so that drafted tokens are counted as if
    they stood.  An entry that occurs in it has a positive logit divided by repetition[s], any other multiplied; one that
    occurs c > 0 times past the first prompt_lens[s] tokens loses c frequency[s] + presence[s].  The lists
    ``bias_tokens`` int32 and ``bias`` float32 [sequences, n] add to the entries that they name (-1: none; of equal ones the
    last).  ``mask`` int32 [rows, ceil(vocab / 32)]: entry x stays where bit x % 32 of word x // 32 is set, and becomes
    -inf elsewhere.  Penalties are float32 [sequences].  Rows of no sequence are not written.  ``out`` may be logits.
    No gradient."""
    if stream is None:
        short = _short or _native()
        got = short and short.adjust(logits, starts, tokens, lens, prompt_lens, repetition, presence, frequency, bias_tokens, bias, mask,
                                     out)
        if got is not None and got is not False:
            return _ended("keops_adjust_logits", got)
    _tensor(logits, "logits"), _tensor(starts, "starts")
    dev, kind = logits.get_device(), _ROWS.get(logits.dtype)
    if logits.dim() != 2 or kind is None or dev < 0 or (logits.shape[1] > 1 and logits.stride(1) != 1):
        raise ValueError("logits must be a bfloat16, float16 or float32 CUDA tensor [rows, vocab] with contiguous rows")
    T, V = logits.shape
    if V < 1:
        raise ValueError("the vocabulary is empty")
    if starts.dim() != 1 or starts.shape[0] < 1:
        raise ValueError("starts must be an int32 tensor [sequences + 1]")
    S = starts.shape[0] - 1
    i32, f32 = torch.int32, torch.float32
    st = _vec(starts, "starts", (S + 1,), i32, dev)
    text = text_stride = width = 0
    if tokens is not None:
        if lens is None:
            raise ValueError("tokens need lens")
        text, text_stride, width = _table(tokens, "tokens", S, dev)
    elif not all(t is None for t in (prompt_lens, repetition, presence, frequency)):
        raise ValueError("penalties need tokens")

    def each(t, name, dtype):
        return 0 if t is None else _vec(t, name, (S,), dtype, dev)
    lp, pp = each(lens, "lens", i32), each(prompt_lens, "prompt_lens", i32)
    rp, ep, fp = each(repetition, "repetition", f32), each(presence, "presence", f32), each(frequency, "frequency", f32)
    ids = add = count = 0
    if (bias_tokens is None) != (bias is None):
        raise ValueError("bias_tokens and bias belong together")
    if bias is not None:
        _tensor(bias_tokens, "bias_tokens")
        if bias_tokens.dim() != 2:
            raise ValueError(f"bias_tokens must be an int32 tensor [{S}, n]")
        count = bias_tokens.shape[1]
        ids, add = _vec(bias_tokens, "bias_tokens", (S, count), i32, dev), _vec(bias, "bias", (S, count), f32, dev)
    mp = mask_stride = 0
    if mask is not None:
        mp, mask_stride, words = _table(mask, "mask", T, dev)
        if words != -(-V // 32):
            raise ValueError(f"mask must have {-(-V // 32)} words a row, got {words}")
    other = _other(stream, dev)
    with torch.cuda.stream(other):
        made = logits.new_empty((T, V)) if out is None else None
    out = made if out is None else _given(out, "out", logits, (T, V))
    if V > 1 and out.stride(1) != 1:
        raise ValueError("out must have contiguous rows")
    rules = _RULES.pack(st, text, text_stride, lp, pp, rp, ep, fp, ids, add, mp, mask_stride, S, width, count)
    _run("keops_adjust_logits", dev, stream, lib().keops_adjust_logits, logits.data_ptr(), logits.stride(0) if T > 1 else V, kind, T, V,
         rules, out.data_ptr(), out.stride(0) if T > 1 else V)
    _keep(other, dev, made)
    if made is None:
        _written(out)
    return out
