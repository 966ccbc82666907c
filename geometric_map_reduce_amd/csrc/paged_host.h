// paged_host.h -- host-side checks that the entry points over a paged cache share.
#pragma once

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "host.h"
#include "keops_mi355x.h"
#include "paged.h"

namespace kmi {

constexpr int64_t kMaxGrid = 0x7fffffff;
// A launch has fewer than 2^32 threads (HIP's limit along an axis).
inline bool launchable(double blocks, int threads) { return blocks * threads < 4294967296.0; }

inline bool aligned(const void *p, uintptr_t to) { return ((uintptr_t)p & (to - 1)) == 0; }

// Bytes of n elements.
inline double bytes_of(int type, double n) { return n * held_bits(type) / 8.0; }
// Bytes of a slot and head's key (or value): its elements and, in 4 bits, their powers.
inline int row_bytes(const keops_cache_t &c) {
  return c.dim * held_bits(c.type) / 8 + (c.type == KEOPS_TYPE_E2M1 ? c.dim / kPowerBlock : 0);
}

// Sizes for the overlap checks: exact where a device could hold them, cut at 2^62.
inline int64_t cut(double bytes) { return bytes < 4.6e18 ? (int64_t)bytes : (int64_t)1 << 62; }

// Bytes from the first to past the last element of the pages.
inline int64_t pages_extent(const keops_cache_t &c) {
  if (c.pages == 0) return 0;
  return cut(bytes_of(c.type, (double)(c.pages - 1) * (double)c.page_stride + (double)(c.page_size - 1) * (double)c.slot_stride +
                                  (double)(c.heads - 1) * (double)c.head_stride + c.dim));
}
// Bytes of the 4-bit blocks' powers of keys, or of values.
inline int64_t powers_extent(const keops_cache_t &c) {
  return c.type == KEOPS_TYPE_E2M1 ? cut((double)c.pages * c.heads * (double)c.page_size * (c.dim / kPowerBlock)) : 0;
}
inline int64_t weights_extent(const keops_cache_t &c) {
  return c.weights ? cut((double)c.pages * c.heads * (double)c.page_size * 4.0) : 0;
}
// Whether `bytes` at p meet the pool: pages, weights or powers.
inline bool meets_cache(const keops_cache_t &c, const void *p, int64_t bytes) {
  const int64_t pb = pages_extent(c), wb = weights_extent(c), eb = powers_extent(c);
  return overlaps(p, bytes, c.k_pages, pb) || overlaps(p, bytes, c.v_pages, pb) || overlaps(p, bytes, c.weights, wb) ||
         overlaps(p, bytes, c.k_powers, eb) || overlaps(p, bytes, c.v_powers, eb);
}
// Bytes of `tokens` rows of `row` 16-bit elements, `stride` apart.
inline int64_t rows_extent(int64_t tokens, int64_t stride, int64_t row) {
  return cut(((double)(tokens - 1) * (double)stride + (double)row) * 2.0);
}
// Elements between 16-bit rows: not negative, whole 16 bytes, within 2^40.
inline bool good_stride(int64_t st) { return st >= 0 && st <= (int64_t)1 << 40 && st % 8 == 0; }

inline int check_cache(const keops_cache_t *c, bool scales = true) {
  if (!c) return KEOPS_ERR_INVALID_ARG;
  if (c->pages < 0 || c->page_size < 1 || c->heads < 1 || c->dim < 1 || c->seqs < 0 || c->table_width < 0 ||
      c->table_stride < 0)
    return KEOPS_ERR_INVALID_ARG;
  if (c->type != KEOPS_TYPE_BF16 && c->type != KEOPS_TYPE_F16 && c->type != KEOPS_TYPE_E4M3 && c->type != KEOPS_TYPE_E2M1)
    return KEOPS_ERR_INVALID_ARG;
  const bool e2m1 = c->type == KEOPS_TYPE_E2M1;
  if (e2m1 && (c->pages > 0 && (!c->k_powers || !c->v_powers))) return KEOPS_ERR_INVALID_ARG;
  if (e2m1 && (!aligned(c->k_powers, 16) || !aligned(c->v_powers, 16))) return KEOPS_ERR_INVALID_ARG;
  if (scales && c->type == KEOPS_TYPE_E4M3 && (!c->k_scale || !c->v_scale)) return KEOPS_ERR_INVALID_ARG;
  if (c->pages > 0 && (!c->k_pages || !c->v_pages)) return KEOPS_ERR_INVALID_ARG;
  for (int64_t st : {c->page_stride, c->slot_stride, c->head_stride})
    if (st < 0 || st > (int64_t)1 << 40 || st % (128 / held_bits(c->type))) return KEOPS_ERR_INVALID_ARG;
  if (!aligned(c->k_pages, 16) || !aligned(c->v_pages, 16)) return KEOPS_ERR_INVALID_ARG;
  for (const void *p : {(const void *)c->weights, (const void *)c->k_scale, (const void *)c->v_scale,
                        (const void *)c->page_table, (const void *)c->lens})
    if (!aligned(p, 4)) return KEOPS_ERR_INVALID_ARG;
  if (c->seqs > 0 && (!c->lens || (c->table_width > 0 && !c->page_table))) return KEOPS_ERR_INVALID_ARG;
  if (c->dim != 64 && c->dim != 96 && c->dim != 128 && c->dim != 256) return KEOPS_ERR_UNSUPPORTED;
  if (c->pages > 0x7fffffff || c->heads > 65535) return KEOPS_ERR_UNSUPPORTED;
  // a slot and head's number, by which the kernels find its powers, has 32 bits
  if (e2m1 && (double)c->pages * c->heads * (double)c->page_size > 4294967295.0) return KEOPS_ERR_UNSUPPORTED;
  return KEOPS_OK;
}

inline CacheView view_of(const keops_cache_t &c) {
  CacheView v{};
  v.k = (char *)c.k_pages;
  v.v = (char *)c.v_pages;
  v.weights = c.weights;
  if (c.type == KEOPS_TYPE_E2M1) {
    v.k_power = c.k_powers;
    v.v_power = c.v_powers;
  } else {
    v.k_scale = c.k_scale;
    v.v_scale = c.v_scale;
  }
  v.page_stride = c.page_stride * held_bits(c.type) / 8;
  v.slot_stride = c.slot_stride * held_bits(c.type) / 8;
  v.head_stride = c.head_stride * held_bits(c.type) / 8;
  v.page = make_fastdiv((uint32_t)c.page_size);
  v.pages = (uint32_t)c.pages;
  v.heads = c.heads;
  v.dim = c.dim;
  v.table = c.page_table;
  v.table_stride = c.table_stride;
  v.table_width = (uint32_t)c.table_width;
  v.lens = c.lens;
  v.seqs = c.seqs;
  return v;
}

inline int64_t align256(int64_t v) { return (v + 255) / 256 * 256; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }


// The type of a call's 16-bit rows beside a cache: the cache's own, any 16-bit one with a narrower cache.
inline bool good_rows_type(const keops_cache_t &c, int type) {
  return (type == KEOPS_TYPE_BF16 || type == KEOPS_TYPE_F16) &&
         (c.type == KEOPS_TYPE_E4M3 || c.type == KEOPS_TYPE_E2M1 || c.type == type);
}

}  // namespace kmi
