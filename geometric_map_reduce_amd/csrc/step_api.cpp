// step_api.cpp -- the C ABI of the operators around the paged cache: rotary positions, the append that
// rotates, reading slots back, and the adjustment of logits.  No HIP call is made before the arguments are
// validated, and no exception leaves an entry point.
#include <hip/hip_runtime.h>

#include "paged_host.h"
#include "step.h"

namespace kmi {
namespace {

// Strides within 2^40 elements: offsets of 2^31 rows stay in 64 bits.
bool small_stride(int64_t st) { return st >= 0 && st <= (int64_t)1 << 40; }

// Bytes from the first element to past the last of `rows` rows of `row` elements.
int64_t span_bytes(int type, int64_t rows, int64_t stride, double row) {
  return rows > 0 ? cut(bytes_of(type, (double)(rows - 1) * (double)stride + row)) : 0;
}

int check_rotary(const keops_rotary_t *r, int64_t dim) {
  if (!r || r->pairs < 0 || !std::isfinite(r->factor)) return KEOPS_ERR_INVALID_ARG;
  if (2 * (int64_t)r->pairs > dim) return KEOPS_ERR_INVALID_ARG;
  if (r->pairs > 0 && (!r->freqs || !aligned(r->freqs, 8))) return KEOPS_ERR_INVALID_ARG;
  return KEOPS_OK;
}

RotaryView rotation_of(const keops_rotary_t &r, bool inverse) {
  return {r.freqs, r.factor, inverse ? -1.0 : 1.0, r.pairs, r.interleaved != 0};
}

constexpr int kRotaryLds = 64 << 10;         // bytes of a work-group's cosines and sines at most

int rotary_entry(const void *x, int64_t x_stride, int type, int64_t tokens, int heads, int dim, const int32_t *positions,
                 const keops_rotary_t *rotary, int inverse, void *out, int64_t out_stride, hipStream_t st) {
  if (type != KEOPS_TYPE_BF16 && type != KEOPS_TYPE_F16 && type != KEOPS_TYPE_F32) return KEOPS_ERR_INVALID_ARG;
  if (tokens < 0 || heads < 0 || dim < 1) return KEOPS_ERR_INVALID_ARG;
  if (int rc = check_rotary(rotary, dim)) return rc;
  if (!small_stride(x_stride) || !small_stride(out_stride)) return KEOPS_ERR_INVALID_ARG;
  const int64_t row = (int64_t)heads * dim;
  const int bytes = held_bits(type) / 8;
  if (tokens > 1 && out_stride < row) return KEOPS_ERR_INVALID_ARG;
  if (tokens > 0 && heads > 0) {
    if (!x || !out || !aligned(x, bytes) || !aligned(out, bytes)) return KEOPS_ERR_INVALID_ARG;
    if (rotary->pairs > 0 && (!positions || !aligned(positions, 4))) return KEOPS_ERR_INVALID_ARG;
    const int64_t xb = span_bytes(type, tokens, x_stride, (double)row), ob = span_bytes(type, tokens, out_stride, (double)row);
    if (overlaps(out, ob, x, xb) && !(x == out && (x_stride == out_stride || tokens == 1))) return KEOPS_ERR_INVALID_ARG;
    if (overlaps(out, ob, positions, cut((double)tokens * 4.0)) || overlaps(out, ob, rotary->freqs, (int64_t)rotary->pairs * 8))
      return KEOPS_ERR_INVALID_ARG;
  }
  if (tokens > 0x7fffffff || heads > 65535 || dim > 65536 || rotary->pairs * (int)sizeof(float2) > kRotaryLds) return KEOPS_ERR_UNSUPPORTED;
  if (tokens == 0 || heads == 0) return KEOPS_OK;
  (void)hipGetLastError();
  RotaryArgs a{};
  a.x = x;
  a.out = out;
  a.x_stride = tokens > 1 ? x_stride : row;
  a.out_stride = tokens > 1 ? out_stride : row;
  a.positions = positions;
  a.r = rotation_of(*rotary, inverse != 0);
  a.tokens = tokens;
  a.heads = heads;
  a.dim = dim;
  // the widest pieces, of up to eight columns and 16 bytes, that everything is made of
  int piece = 16 / bytes;
  while (piece > 1 && (a.r.pairs % piece || dim % piece || !aligned(x, piece * bytes) || !aligned(out, piece * bytes) ||
                       a.x_stride % piece || a.out_stride % piece))
    piece /= 2;
  const bool copies = x != out;
  a.pieces = a.r.pairs / piece + (copies ? (dim - 2 * a.r.pairs) / piece : 0);
  if (a.pieces == 0) return KEOPS_OK;        // in place, and nothing turns
  int cus = 0;
  if (int rc = device_setup(&cus)) return rc;
  // tokens of a work-group: a cosine for each thread, as long as the device is full
  const int pairs = std::max(a.r.pairs, 1);
  int64_t per = std::max(1, kRotaryThreads / pairs);
  per = std::max<int64_t>(1, std::min(per, tokens / (4 * cus)));
  per = std::min(per, std::max<int64_t>(1, ((int64_t)1 << 30) / ((int64_t)heads * a.pieces)));
  a.tokens_wg = (int)per;
  a.pairs_div = make_fastdiv((uint32_t)pairs);
  a.pieces_div = make_fastdiv((uint32_t)a.pieces);
  a.heads_div = make_fastdiv((uint32_t)heads);
  const int64_t groups = ceil_div(tokens, per), items = per * heads * a.pieces;
  if (items > 0x7fffffff - 65536 * kRotaryThreads) return KEOPS_ERR_UNSUPPORTED;
  const int64_t shares = std::max<int64_t>(1, std::min({ceil_div(items, kRotaryThreads), ceil_div(4 * cus, groups), (int64_t)65535}));
  if (!launchable((double)groups, kRotaryThreads)) return KEOPS_ERR_UNSUPPORTED;
  launch_rotary(a, type, piece, dim3((unsigned)groups, (unsigned)shares), st);
  return check_launch();
}

int append_rotary_entry(const keops_cache_t *c, const void *q, const void *k, const void *v, int64_t q_stride, int64_t k_stride,
                        int64_t v_stride, int type, int heads, const int32_t *starts, int64_t tokens, const int32_t *positions,
                        const keops_rotary_t *rotary, void *q_out, int64_t q_out_stride, hipStream_t st) {
  if (int rc = check_cache(c)) return rc;
  if (!good_rows_type(*c, type)) return KEOPS_ERR_INVALID_ARG;
  if (tokens < 0 || heads < 0) return KEOPS_ERR_INVALID_ARG;
  if (int rc = check_rotary(rotary, c->dim)) return rc;
  if (heads > 65535) return KEOPS_ERR_UNSUPPORTED;
  const int64_t row = (int64_t)c->heads * c->dim, qrow = (int64_t)heads * c->dim;
  if (tokens > 0) {
    if (!k || !v || !aligned(k, 16) || !aligned(v, 16) || !good_stride(k_stride) || !good_stride(v_stride)) return KEOPS_ERR_INVALID_ARG;
    if (heads > 0 && (!q || !q_out || !aligned(q, 16) || !aligned(q_out, 16) || !good_stride(q_stride) || !good_stride(q_out_stride)))
      return KEOPS_ERR_INVALID_ARG;
    if (heads > 0 && tokens > 1 && q_out_stride < qrow) return KEOPS_ERR_INVALID_ARG;
    if (c->seqs > 0 && (!starts || !aligned(starts, 4))) return KEOPS_ERR_INVALID_ARG;
    if (!aligned(positions, 4)) return KEOPS_ERR_INVALID_ARG;
    const int64_t kb = rows_extent(tokens, k_stride, row), vb = rows_extent(tokens, v_stride, row);
    const int64_t qb = heads > 0 ? rows_extent(tokens, q_stride, qrow) : 0, ob = heads > 0 ? rows_extent(tokens, q_out_stride, qrow) : 0;
    const struct { const void *p; int64_t bytes; } inputs[] = {{k, kb}, {v, vb}, {q, qb}, {positions, positions ? cut((double)tokens * 4.0) : 0},
                                                              {rotary->freqs, (int64_t)rotary->pairs * 8}};
    for (const auto &in : inputs)
      if (meets_cache(*c, in.p, in.bytes) || overlaps(q_out, ob, in.p, in.bytes)) return KEOPS_ERR_INVALID_ARG;
    if (meets_cache(*c, q_out, ob)) return KEOPS_ERR_INVALID_ARG;
  }
  const double pieces = (double)(qrow + 2 * row) / 8.0;
  if (tokens > 0x7fffffff || pieces > (double)(1 << 28) || !launchable((double)tokens, kTurnThreads)) return KEOPS_ERR_UNSUPPORTED;
  if (tokens == 0 || c->seqs == 0) return KEOPS_OK;
  (void)hipGetLastError();
  int cus = 0;
  if (int rc = device_setup(&cus)) return rc;
  AppendRotaryArgs a{};
  a.c = view_of(*c);
  a.q = (const char *)q;
  a.k = (const char *)k;
  a.v = (const char *)v;
  a.q_out = (char *)q_out;
  a.q_stride = q_stride * 2;
  a.k_stride = k_stride * 2;
  a.v_stride = v_stride * 2;
  a.q_out_stride = q_out_stride * 2;
  a.starts = starts;
  a.positions = positions;
  a.r = rotation_of(*rotary, false);
  a.tokens = tokens;
  a.heads = heads;
  // tokens of a work-group: as many as there are waves to look for their slots, as long as the device is full
  a.tokens_wg = (int)std::max<int64_t>(1, std::min<int64_t>(kTurnTokens, tokens / (4 * cus)));
  a.items_div = make_fastdiv((uint32_t)((qrow + 2 * row) / 8));
  a.dim_div = make_fastdiv((uint32_t)(c->dim / 8));
  const int64_t groups = ceil_div(tokens, a.tokens_wg), items = a.tokens_wg * ((qrow + 2 * row) / 8);
  const int64_t shares = std::max<int64_t>(1, std::min({ceil_div(items, kTurnThreads), ceil_div(4 * cus, groups), (int64_t)65535}));
  launch_append_rotary(a, type, held_bits(c->type), dim3((unsigned)groups, (unsigned)shares), st);
  return check_launch();
}

int read_entry(const keops_cache_t *c, void *k, void *v, int64_t k_stride, int64_t v_stride, int type, const int32_t *starts,
               int64_t tokens, hipStream_t st) {
  if (int rc = check_cache(c)) return rc;
  if (!good_rows_type(*c, type)) return KEOPS_ERR_INVALID_ARG;
  if (tokens < 0) return KEOPS_ERR_INVALID_ARG;
  const int64_t row = (int64_t)c->heads * c->dim;
  if (tokens > 0) {
    if (!k || !v || !aligned(k, 16) || !aligned(v, 16) || !good_stride(k_stride) || !good_stride(v_stride)) return KEOPS_ERR_INVALID_ARG;
    if (tokens > 1 && (k_stride < row || v_stride < row)) return KEOPS_ERR_INVALID_ARG;
    if (c->seqs > 0 && (!starts || !aligned(starts, 4))) return KEOPS_ERR_INVALID_ARG;
    const int64_t kb = rows_extent(tokens, k_stride, row), vb = rows_extent(tokens, v_stride, row);
    // keys and values may alternate in the rows of one array
    const bool rows_apart = k_stride == v_stride && std::max((uintptr_t)k, (uintptr_t)v) - std::min((uintptr_t)k, (uintptr_t)v) >= (uintptr_t)(row * 2) &&
                            (double)(std::max((uintptr_t)k, (uintptr_t)v) - std::min((uintptr_t)k, (uintptr_t)v)) + (double)row * 2 <= (double)k_stride * 2;
    if (overlaps(k, kb, v, vb) && !(tokens > 1 && rows_apart)) return KEOPS_ERR_INVALID_ARG;
    if (meets_cache(*c, k, kb) || meets_cache(*c, v, vb)) return KEOPS_ERR_INVALID_ARG;
  }
  if (tokens > 0x7fffffff || !launchable(std::ceil((double)tokens * (double)(row / 8) / 256.0), 256)) return KEOPS_ERR_UNSUPPORTED;
  if (tokens == 0 || c->seqs == 0) return KEOPS_OK;
  (void)hipGetLastError();
  ReadArgs a{};
  a.c = view_of(*c);
  a.k = (char *)k;
  a.v = (char *)v;
  a.k_stride = k_stride * 2;
  a.v_stride = v_stride * 2;
  a.starts = starts;
  a.tokens = tokens;
  launch_read(a, type, held_bits(c->type), st);
  return check_launch();
}

int logits_entry(const void *logits, int64_t stride, int type, int64_t rows, int vocab, const keops_logit_rules_t *r, void *out,
                 int64_t out_stride, hipStream_t st) {
  if (type != KEOPS_TYPE_BF16 && type != KEOPS_TYPE_F16 && type != KEOPS_TYPE_F32) return KEOPS_ERR_INVALID_ARG;
  if (!r || rows < 0 || vocab < 1 || r->seqs < 0 || r->text_width < 0 || r->biases < 0) return KEOPS_ERR_INVALID_ARG;
  if (!small_stride(stride) || !small_stride(out_stride) || !small_stride(r->mask_stride) || !small_stride(r->text_stride))
    return KEOPS_ERR_INVALID_ARG;
  const int bytes = held_bits(type) / 8;
  const int64_t words = ceil_div(vocab, 32);
  for (const void *p : {(const void *)r->starts, (const void *)r->text, (const void *)r->lens, (const void *)r->prompt_lens,
                        (const void *)r->repetition, (const void *)r->presence, (const void *)r->frequency,
                        (const void *)r->bias_tokens, (const void *)r->bias, (const void *)r->mask})
    if (!aligned(p, 4)) return KEOPS_ERR_INVALID_ARG;
  if (rows > 0 && r->seqs > 0) {
    if (!logits || !out || !aligned(logits, bytes) || !aligned(out, bytes) || !r->starts) return KEOPS_ERR_INVALID_ARG;
    if (rows > 1 && out_stride < vocab) return KEOPS_ERR_INVALID_ARG;
    if (r->text && !r->lens) return KEOPS_ERR_INVALID_ARG;
    if (r->biases > 0 && (!r->bias_tokens || !r->bias)) return KEOPS_ERR_INVALID_ARG;
    const int64_t lb = span_bytes(type, rows, stride, vocab), ob = span_bytes(type, rows, out_stride, vocab);
    if (overlaps(out, ob, logits, lb) && !(out == logits && (stride == out_stride || rows == 1))) return KEOPS_ERR_INVALID_ARG;
    const int64_t sb = (int64_t)r->seqs * 4, bb = cut((double)r->seqs * r->biases * 4.0);
    const struct { const void *p; int64_t bytes; } inputs[] = {
        {r->starts, sb + 4}, {r->lens, sb}, {r->prompt_lens, sb}, {r->repetition, sb}, {r->presence, sb}, {r->frequency, sb},
        {r->bias_tokens, bb}, {r->bias, bb},
        {r->text, r->text ? span_bytes(KEOPS_TYPE_F32, r->seqs, r->text_stride, r->text_width) : 0},
        {r->mask, r->mask ? span_bytes(KEOPS_TYPE_F32, rows, r->mask_stride, (double)words) : 0}};
    for (const auto &in : inputs)
      if (in.p && overlaps(out, ob, in.p, in.bytes)) return KEOPS_ERR_INVALID_ARG;
  }
  if (rows > 0x7fffffff || vocab > 1 << 30 || r->text_width >= 1 << 30 || r->biases > 1 << 30)
    return KEOPS_ERR_UNSUPPORTED;
  if (rows == 0 || r->seqs == 0) return KEOPS_OK;
  LogitArgs a{};
  a.logits = logits;
  a.out = out;
  a.stride = rows > 1 ? stride : 0;
  a.out_stride = rows > 1 ? out_stride : 0;
  a.rows = rows;
  a.vocab = vocab;
  a.starts = r->starts;
  a.text = r->text_width > 0 ? r->text : nullptr;
  a.lens = r->lens;
  a.prompt_lens = r->prompt_lens;
  a.text_stride = r->text_stride;
  a.repetition = r->repetition;
  a.presence = r->presence;
  a.frequency = r->frequency;
  a.bias_tokens = r->bias_tokens;
  a.bias = r->bias;
  a.mask = (const uint32_t *)r->mask;
  a.mask_stride = rows > 1 ? r->mask_stride : 0;
  a.seqs = r->seqs;
  a.text_width = r->text_width;
  a.biases = r->biases;
  const int to = 16 / bytes;
  a.whole = aligned(logits, 16) && aligned(out, 16) && a.stride % to == 0 && a.out_stride % to == 0;
  a.piece = (double)rows * (double)ceil_div(vocab, kLogitPiece) >= 256.0 ? kLogitPiece : kLogitPiece / 2;
  a.pieces_inverse = 1.0f / (float)ceil_div(vocab, a.piece);
  const double blocks = (double)rows * (double)ceil_div(vocab, a.piece);
  if (blocks > (double)kMaxGrid || !launchable(blocks, kLogitThreads)) return KEOPS_ERR_UNSUPPORTED;
  (void)hipGetLastError();
  launch_adjust_logits(a, type, dim3((unsigned)blocks), st);
  return check_launch();
}

}  // namespace
}  // namespace kmi

using namespace kmi;

extern "C" {

int keops_rotary(const void *x, int64_t x_stride, int32_t type, int64_t tokens, int32_t heads, int32_t dim,
                 const int32_t *positions, const keops_rotary_t *rotary, int32_t inverse, void *out, int64_t out_stride,
                 void *stream) {
  try {
    return rotary_entry(x, x_stride, type, tokens, heads, dim, positions, rotary, inverse, out, out_stride, (hipStream_t)stream);
  } catch (...) {
    return KEOPS_ERR_ALLOC;
  }
}

int keops_cache_append_rotary(const keops_cache_t *cache, const void *q, const void *k, const void *v, int64_t q_stride,
                              int64_t k_stride, int64_t v_stride, int32_t type, int32_t heads, const int32_t *starts,
                              int64_t tokens, const int32_t *positions, const keops_rotary_t *rotary, void *q_out,
                              int64_t q_out_stride, void *stream) {
  try {
    return append_rotary_entry(cache, q, k, v, q_stride, k_stride, v_stride, type, heads, starts, tokens, positions, rotary, q_out,
                               q_out_stride, (hipStream_t)stream);
  } catch (...) {
    return KEOPS_ERR_ALLOC;
  }
}

int keops_cache_read(const keops_cache_t *cache, void *k, void *v, int64_t k_stride, int64_t v_stride, int32_t type,
                     const int32_t *starts, int64_t tokens, void *stream) {
  try {
    return read_entry(cache, k, v, k_stride, v_stride, type, starts, tokens, (hipStream_t)stream);
  } catch (...) {
    return KEOPS_ERR_ALLOC;
  }
}

int keops_adjust_logits(const void *logits, int64_t stride, int32_t type, int64_t rows, int32_t vocab,
                        const keops_logit_rules_t *rules, void *out, int64_t out_stride, void *stream) {
  try {
    return logits_entry(logits, stride, type, rows, vocab, rules, out, out_stride, (hipStream_t)stream);
  } catch (...) {
    return KEOPS_ERR_ALLOC;
  }
}

}  // extern "C"
