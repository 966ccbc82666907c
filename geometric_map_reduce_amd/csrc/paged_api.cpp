// paged_api.cpp -- the C ABI of the paged key/value cache and of draft verification:
// argument validation, launch plans and workspace.  No HIP call is made before the
// arguments are validated, and no exception leaves an entry point.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "host.h"
#include "keops_mi355x.h"
#include "paged.h"

namespace kmi {
namespace {

constexpr int64_t kMaxGrid = 0x7fffffff;
// A launch has fewer than 2^32 threads (HIP's limit along an axis).
bool launchable(double blocks, int threads) { return blocks * threads < 4294967296.0; }
constexpr int64_t kMaxBlocks = (1 << 24) - 1;    // of 256 threads
constexpr double kMaxWorkspace = 1.0e14;    // more than any device holds; below the 64-bit limit
// Work-groups that a launch aims for, per compute unit, when it splits a long axis.
constexpr int64_t kManyWgsPerCu = 2;
constexpr int64_t kSumsWgsPerCu = 6;    // 4: 276 to 266 us for 36 prompts with a window, 1,056 to 1,012 for 4,096 tokens (dim 64)
// Few rows: least slots of a work-group's run (one tile of 32 for each wave), and the longest
// sequences that are left whole when there are enough of them to fill the device.
constexpr int kFewLeast = 128;
constexpr int kFewWhole = 1024;
// Up to here work-groups of eight waves that have a head's slots to themselves beat splitting them and
// a second pass: 15.6 to 19 us a call at 300 and 600 slots, 18.2 to 18.5 at 1,000, 28.5 to 20.6 at 2,000
// (one compute unit reads at most some 50 bytes a nanosecond).
constexpr int kFewWhole8 = 768;

// Parts of a row from which on its join is shared by columns: 400 parts (one head's 51,206 slots) take 22.6 us
// a call unshared and 19.6 shared, 196 parts 16.8 and 16.4, 128 parts 31.6 and 33.1 (four heads').
constexpr int64_t kJoinParts = 192;
// Keys and values that a call reads at most, in bytes, from which on they pass the caches by.  The last level holds
// 256 MB: 525 MB took 107 us by way of it and 98 past it, and 230 MB that it still held from the call before 47
// and 51 us.  Lengths may fall short of their bound, so not at 256 MB itself.
constexpr double kFarBytes = 384e6;

// Kept scores take 4 bytes a row and slot of the call's bounds, which may lie far above its lengths; a slot's are
// a quarter of its key and value at most, so more than twice the pool means bounds of eight times what it holds.
// Past that, and past 4 GB, the weights come from the column sums instead, which need no scores.  They cost 64
// sequences of 4,000 slots (4 rows, 8 heads of 128, bounds of 131,072) 474 us in place of 311, 16 of 20,000 slots
// (32 rows) 462 in place of 604.  Up to half a GB is a five-hundredth of the device's memory, and always taken.
constexpr double kScoresAlways = 512e6, kScoresMost = 4294967296.0;

bool aligned(const void *p, uintptr_t to) { return ((uintptr_t)p & (to - 1)) == 0; }

int64_t width_of(int type) { return type == KEOPS_TYPE_E4M3 ? 1 : 2; }

// Sizes for the overlap checks: exact where a device could hold them, cut at 2^62.
int64_t cut(double bytes) { return bytes < 4.6e18 ? (int64_t)bytes : (int64_t)1 << 62; }

// Bytes from the first to past the last element of the pages.
int64_t pages_extent(const keops_cache_t &c) {
  if (c.pages == 0) return 0;
  const int64_t w = width_of(c.type);
  return cut(((double)(c.pages - 1) * (double)c.page_stride + (double)(c.page_size - 1) * (double)c.slot_stride +
              (double)(c.heads - 1) * (double)c.head_stride + c.dim) * (double)w);
}
int64_t weights_extent(const keops_cache_t &c) {
  return c.weights ? cut((double)c.pages * c.heads * (double)c.page_size * 4.0) : 0;
}
// Bytes of `tokens` rows of `row` 16-bit elements, `stride` apart.
int64_t rows_extent(int64_t tokens, int64_t stride, int64_t row) {
  return cut(((double)(tokens - 1) * (double)stride + (double)row) * 2.0);
}
// Elements between 16-bit rows: not negative, whole 16 bytes, within 2^40.
bool good_stride(int64_t st) { return st >= 0 && st <= (int64_t)1 << 40 && st % 8 == 0; }

int check_cache(const keops_cache_t *c, bool scales = true) {
  if (!c) return KEOPS_ERR_INVALID_ARG;
  if (c->pages < 0 || c->page_size < 1 || c->heads < 1 || c->dim < 1 || c->seqs < 0 || c->table_width < 0 ||
      c->table_stride < 0)
    return KEOPS_ERR_INVALID_ARG;
  if (c->type != KEOPS_TYPE_BF16 && c->type != KEOPS_TYPE_F16 && c->type != KEOPS_TYPE_E4M3) return KEOPS_ERR_INVALID_ARG;
  if (scales && c->type == KEOPS_TYPE_E4M3 && (!c->k_scale || !c->v_scale)) return KEOPS_ERR_INVALID_ARG;
  if (c->pages > 0 && (!c->k_pages || !c->v_pages)) return KEOPS_ERR_INVALID_ARG;
  const int64_t w = width_of(c->type);
  for (int64_t st : {c->page_stride, c->slot_stride, c->head_stride})
    if (st < 0 || st > (int64_t)1 << 40 || st * w % 16) return KEOPS_ERR_INVALID_ARG;
  if (!aligned(c->k_pages, 16) || !aligned(c->v_pages, 16)) return KEOPS_ERR_INVALID_ARG;
  for (const void *p : {(const void *)c->weights, (const void *)c->k_scale, (const void *)c->v_scale,
                        (const void *)c->page_table, (const void *)c->lens})
    if (!aligned(p, 4)) return KEOPS_ERR_INVALID_ARG;
  if (c->seqs > 0 && (!c->lens || (c->table_width > 0 && !c->page_table))) return KEOPS_ERR_INVALID_ARG;
  if (c->dim != 64 && c->dim != 96 && c->dim != 128 && c->dim != 256) return KEOPS_ERR_UNSUPPORTED;
  if (c->pages > 0x7fffffff || c->heads > 65535) return KEOPS_ERR_UNSUPPORTED;
  return KEOPS_OK;
}

CacheView view_of(const keops_cache_t &c) {
  const int64_t w = width_of(c.type);
  CacheView v{};
  v.k = (char *)c.k_pages;
  v.v = (char *)c.v_pages;
  v.weights = c.weights;
  v.k_scale = c.k_scale;
  v.v_scale = c.v_scale;
  v.page_stride = c.page_stride * w;
  v.slot_stride = c.slot_stride * w;
  v.head_stride = c.head_stride * w;
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

int64_t align256(int64_t v) { return (v + 255) / 256 * 256; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Launch plan of one attention call.
struct AttendPlan {
  bool few, scores, far;
  int whole, row_tiles, score_rows, join_rows, join_slices;
  int64_t nsplit, nrow, grid, sums_grid, score_stride;
  int64_t line_bytes, ml_bytes, o_bytes, score_bytes, sums_bytes;
  int64_t total() const { return line_bytes + ml_bytes + o_bytes + score_bytes + sums_bytes; }
};

int plan_attend(const keops_cache_t &c, int type, int64_t tokens, int heads, int64_t max_q, int64_t max_len, int window, int cus,
                AttendPlan *p) {
  *p = AttendPlan{};
  const int64_t G = heads / c.heads, rows = max_q * G, S = c.seqs, H = c.heads;
  p->few = rows <= kFewRowsMax;
  // keeping a row's scores costs 8 bytes a slot, reading K again dim times its width
  const double heads_of_seqs = (double)S * (double)H;
  const double score_bytes = 4.0 * heads_of_seqs * (double)rows * (double)(ceil_div(max_len, 32) * 32);
  const double pool_bytes = 2.0 * (double)c.pages * c.page_size * (double)H * (double)(c.dim * width_of(c.type));
  const bool sums_fit = heads_of_seqs * (double)ceil_div(max_len, kSumSlotsTile) <= (double)kMaxGrid / 1024;
  p->scores = c.weights && p->few && rows * 8 <= c.dim * width_of(c.type) &&
              (score_bytes <= std::max(kScoresAlways, std::min(2.0 * pool_bytes, kScoresMost)) || !sums_fit);
  // slots that the rows of one sequence see at most
  int64_t span = max_len;
  if (window > 0) span = std::min<int64_t>(span, (int64_t)window + max_q - 1);
  if (p->few) {
    p->row_tiles = rows <= 16 ? 1 : 2;
    const int64_t from_tile = std::min<int64_t>(max_len, span + 31);    // a window starts inside a tile
    if ((double)S * (double)H * (double)(from_tile / 32 + 2) > (double)kMaxGrid || (double)S * (double)H * (double)rows * 8.0 > (double)kMaxGrid)
      return KEOPS_ERR_UNSUPPORTED;
    AttendArgs probe{};
    probe.score_stride = p->scores;
    const int fit = launch_attend_few(probe, type, c.type == KEOPS_TYPE_E4M3, c.dim, p->row_tiles, 0, 0, nullptr);
    if (fit < 1) return KEOPS_ERR_HIP;
    const int64_t room = (int64_t)fit * cus;
    p->whole = rows == 0 || from_tile <= kFewLeast || (from_tile <= kFewWhole && S * H * 2 >= room);
    if (!p->whole && from_tile <= kFewWhole8 && S * H <= cus && p->row_tiles == 1 && c.dim <= 128) p->whole = 2;
    if (p->whole && !launchable((double)S * (double)H, p->whole == 2 ? 512 : 256)) return KEOPS_ERR_UNSUPPORTED;
    p->grid = p->whole ? S * H : std::min(room, ceil_div(S * H * from_tile, kFewLeast));
    p->far = !p->whole && 2.0 * (double)S * (double)H * (double)from_tile * (double)(c.dim * width_of(c.type)) > kFarBytes;
    if (!p->whole) {
      // a joining work-group's 1024 / dim groups of threads: one to a row where the parts are few
      const int64_t groups = 1024 / c.dim, parts = ceil_div(p->grid, S * H) + 1;
      p->join_rows = (int)std::max<int64_t>(1, std::min(rows, parts <= 4 ? groups : groups / parts));
      // many parts: 32 columns to a work-group, so that 32 groups of threads share a row's parts
      p->join_slices = parts > kJoinParts ? c.dim / 32 : 1;
      p->line_bytes = align256((S + 1) * 4);
      p->ml_bytes = align256(p->grid * 2 * 16 * p->row_tiles * 8);
      p->o_bytes = align256(p->grid * 2 * 16 * p->row_tiles * c.dim * 4);
    }
  } else {
    const int64_t nrt = ceil_div(rows, kManyRowsTile);
    if ((double)S * (double)H * (double)nrt > (double)kMaxGrid / 1024) return KEOPS_ERR_UNSUPPORTED;
    const int64_t wgs = S * H * nrt;
    // as many splits as the device holds at once, of at least four tiles of slots
    const int64_t room = (c.dim > 128 ? 1 : kManyWgsPerCu) * cus;
    p->nsplit = std::max<int64_t>(1, std::min(room / wgs, span / 256));
    // the join looks through all tokens' rows
    if (p->nsplit > 1 && !launchable((double)join_blocks(tokens * heads, c.dim, (int)p->nsplit), kJoinThreads)) p->nsplit = 1;
    p->grid = wgs * p->nsplit;
  }
  if (c.weights) {
    if (p->scores) {
      p->score_rows = (int)rows;
      p->score_stride = ceil_div(max_len, 32) * 32;
      if (score_bytes > kMaxWorkspace) return KEOPS_ERR_ALLOC;
      p->score_bytes = align256(4 * S * H * rows * p->score_stride);
    } else {
      const int64_t nst = ceil_div(max_len, kSumSlotsTile);
      if (!sums_fit) return KEOPS_ERR_UNSUPPORTED;
      const int64_t wgs = S * H * nst;
      // slots outside every window cost next to nothing
      const int64_t busy = std::max<int64_t>(1, S * H * std::min(nst, ceil_div(span, kSumSlotsTile) + 1));
      p->nrow = std::max<int64_t>(1, std::min({ceil_div(kSumsWgsPerCu * cus, busy), rows / 256, kMaxBlocks / std::max<int64_t>(1, wgs)}));
      p->sums_grid = wgs * p->nrow;
      if (p->nrow > 1) {
        if (4.0 * (double)p->nrow * (double)S * (double)H * (double)max_len > kMaxWorkspace) return KEOPS_ERR_ALLOC;
        p->sums_bytes = align256(4 * p->nrow * S * H * max_len);
      }
    }
  }
  if (p->few) {
    const double joins = p->join_rows ? heads_of_seqs * (double)ceil_div(rows, p->join_rows) * p->join_slices : 0.0;
    const double sums = p->scores ? heads_of_seqs * (double)ceil_div(max_len, kScoreSlots) : 0.0;
    if (!launchable(joins + sums, kFinishThreads)) return KEOPS_ERR_UNSUPPORTED;
  }
  if (!p->few && p->nsplit > 1) {
    const double out_rows = (double)tokens * heads * (double)p->nsplit;
    if (out_rows * c.dim * 4.0 > kMaxWorkspace) return KEOPS_ERR_ALLOC;
    p->ml_bytes = align256(p->nsplit * tokens * heads * 8);
    p->o_bytes = align256(p->nsplit * tokens * heads * c.dim * 4);
  }
  return KEOPS_OK;
}

int check_attend(const keops_cache_t *c, int type, int64_t tokens, int heads, int max_q, int max_len, float scale,
                 int window, float decay) {
  if (int rc = check_cache(c)) return rc;
  if (type != KEOPS_TYPE_BF16 && type != KEOPS_TYPE_F16) return KEOPS_ERR_INVALID_ARG;
  if (c->type != KEOPS_TYPE_E4M3 && c->type != type) return KEOPS_ERR_INVALID_ARG;
  if (tokens < 0 || heads < 1 || heads % c->heads || max_q < 0 || max_len < 0 || window < 0) return KEOPS_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !std::isfinite(decay)) return KEOPS_ERR_INVALID_ARG;
  if (tokens > 0x7fffffff || heads > 65535 || (int64_t)max_q * (heads / c->heads) > 0x3fffffff ||
      max_len > kMaxSlots)
    return KEOPS_ERR_UNSUPPORTED;
  return KEOPS_OK;
}

// Whether a call has work: tokens that count, or, without any, weights that decay all the same.
bool has_work(const keops_cache_t &c, int64_t tokens, int max_q) {
  return c.seqs > 0 && ((tokens > 0 && max_q > 0) || (c.weights && c.pages > 0));
}

// The caller's workspace, or the library's; the library's is never recorded into a graph,
// whose replays could outlive it.
int take_workspace(Workspace &own, void *given, int64_t given_bytes, int64_t need, hipStream_t st, char **ptr) {
  *ptr = nullptr;
  if (need == 0) return KEOPS_OK;
  if (given) {
    if (given_bytes < need) return KEOPS_ERR_SCRATCH;
    *ptr = (char *)given;
    return KEOPS_OK;
  }
  hipStreamCaptureStatus cap = hipStreamCaptureStatusNone;
  if (hipStreamIsCapturing(st, &cap) != hipSuccess) {
    (void)hipGetLastError();
    return KEOPS_ERR_HIP;
  }
  if (cap != hipStreamCaptureStatusNone) return KEOPS_ERR_ALLOC;
  if (int rc = own.acquire(st, 0, (size_t)need)) return rc;
  *ptr = own.ptr();
  return KEOPS_OK;
}

int append_entry(const keops_cache_t *c, const void *k, const void *v, int64_t k_stride, int64_t v_stride, int type,
                 const int32_t *starts, int64_t tokens, hipStream_t st) {
  if (int rc = check_cache(c)) return rc;
  if (type != KEOPS_TYPE_BF16 && type != KEOPS_TYPE_F16) return KEOPS_ERR_INVALID_ARG;
  if (c->type != KEOPS_TYPE_E4M3 && c->type != type) return KEOPS_ERR_INVALID_ARG;
  if (tokens < 0) return KEOPS_ERR_INVALID_ARG;
  const int64_t row = (int64_t)c->heads * c->dim;
  if (tokens > 0 && (!k || !v || !aligned(k, 16) || !aligned(v, 16) || !good_stride(k_stride) || !good_stride(v_stride)))
    return KEOPS_ERR_INVALID_ARG;
  if (tokens > 0 && c->seqs > 0 && (!starts || !aligned(starts, 4))) return KEOPS_ERR_INVALID_ARG;
  if (tokens > 0x7fffffff || !launchable(std::ceil((double)tokens * (double)(row / 8) / 256.0), 256)) return KEOPS_ERR_UNSUPPORTED;
  if (tokens > 0) {
    const int64_t kb = rows_extent(tokens, k_stride, row), vb = rows_extent(tokens, v_stride, row);
    const int64_t pb = pages_extent(*c);
    for (const void *p : {(const void *)c->k_pages, (const void *)c->v_pages})
      if (overlaps(p, pb, k, kb) || overlaps(p, pb, v, vb)) return KEOPS_ERR_INVALID_ARG;
  }
  if (tokens == 0 || c->seqs == 0 || c->pages == 0 || c->table_width == 0) return KEOPS_OK;
  (void)hipGetLastError();
  AppendArgs a{};
  a.c = view_of(*c);
  a.k = (const char *)k;
  a.v = (const char *)v;
  a.k_stride = k_stride * 2;
  a.v_stride = v_stride * 2;
  a.starts = starts;
  a.tokens = tokens;
  launch_append(a, type, c->type, st);
  return check_launch();
}

int attend_entry(const keops_cache_t *c, const void *q, int64_t q_stride, int type, int heads, const int32_t *starts,
                 int64_t tokens, int max_q, int max_len, float scale, int window, float decay, void *out, float *lse,
                 void *workspace, int64_t workspace_bytes, hipStream_t st) {
  if (int rc = check_attend(c, type, tokens, heads, max_q, max_len, scale, window, decay)) return rc;
  const int64_t row = (int64_t)heads * c->dim;
  if (tokens > 0) {
    if (!q || !out || !lse || !aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4) || !good_stride(q_stride))
      return KEOPS_ERR_INVALID_ARG;
    if (c->seqs > 0 && (!starts || !aligned(starts, 4))) return KEOPS_ERR_INVALID_ARG;
    const int64_t ob = tokens * row * 2, lb = tokens * heads * 4, qb = rows_extent(tokens, q_stride, row);
    const int64_t pb = pages_extent(*c), wb = weights_extent(*c);
    if (overlaps(out, ob, q, qb) || overlaps(out, ob, lse, lb) || overlaps(lse, lb, q, qb) ||
        overlaps(out, ob, c->k_pages, pb) || overlaps(out, ob, c->v_pages, pb) || overlaps(out, ob, c->weights, wb) ||
        overlaps(lse, lb, c->weights, wb) || overlaps(lse, lb, c->k_pages, pb) || overlaps(lse, lb, c->v_pages, pb))
      return KEOPS_ERR_INVALID_ARG;
  }
  if (workspace && (!aligned(workspace, 256) || workspace_bytes < 0)) return KEOPS_ERR_INVALID_ARG;
  if (!has_work(*c, tokens, max_q)) return KEOPS_OK;
  if (c->pages == 0) return KEOPS_ERR_INVALID_ARG;    // nothing to address
  if (!starts || !aligned(starts, 4)) return KEOPS_ERR_INVALID_ARG;
  if (tokens == 0) max_q = 0;
  (void)hipGetLastError();
  int cus = 0;
  if (int rc = device_setup(&cus)) return rc;
  AttendPlan p;
  if (int rc = plan_attend(*c, type, tokens, heads, max_q, max_len, window, cus, &p)) return rc;
  Workspace own;
  char *ws = nullptr;
  if (int rc = take_workspace(own, workspace, workspace_bytes, p.total(), st, &ws)) return rc;

  AttendArgs a{};
  a.c = view_of(*c);
  a.q = (const char *)q;
  a.q_stride = q_stride * 2;
  a.starts = starts;
  a.tokens = tokens;
  a.group = heads / c->heads;
  a.gdiv = make_fastdiv((uint32_t)a.group);
  a.max_q = max_q;
  a.max_len = max_len;
  a.window = std::min(window, kMaxSlots);
  a.scale_log2 = scale * kLog2e;
  a.decay = decay;
  a.out = (char *)out;
  a.lse = lse;
  a.nsplit = (int32_t)p.nsplit;
  a.whole = p.whole;
  a.far = p.far;
  a.join_slices = std::max(1, p.join_slices);
  a.line = (uint32_t *)ws;
  ws += p.line_bytes;
  a.part_ml = (float2 *)ws;
  a.part_o = (float *)(ws + p.ml_bytes);
  a.scores = p.scores ? (float *)(ws + p.ml_bytes + p.o_bytes) : nullptr;
  a.score_stride = p.score_stride;
  a.score_rows = p.score_rows;
  a.nrow = (int32_t)std::max<int64_t>(1, p.nrow);
  a.part_w = (float *)(ws + p.ml_bytes + p.o_bytes + p.score_bytes);
  const bool e4m3 = c->type == KEOPS_TYPE_E4M3;
  const int prof = prof_begin(st);
  if (p.few) launch_attend_few(a, type, e4m3, c->dim, p.row_tiles, (int)p.grid, p.join_rows, st);
  else launch_attend_many(a, type, e4m3, c->dim, dim3((unsigned)p.grid), st);
  prof_end(prof, st);
  if (!p.few && p.nsplit > 1) launch_attend_join(a, type, st);
  if (c->weights && max_len > 0 && !p.scores) {
    launch_attend_sums(a, type, e4m3, c->dim, dim3((unsigned)p.sums_grid), st);
    if (p.nrow > 1) launch_attend_sums_join(a, st);
  }
  return check_launch();
}

int evict_entry(const keops_cache_t *c, const int32_t *new_table, int64_t new_stride, int new_width, int budget,
                int sink, int recent, int32_t *kept, int32_t *new_lens, hipStream_t st) {
  if (int rc = check_cache(c, false)) return rc;   // the move copies held values
  if (budget < 1 || sink < 0 || recent < 0 || (int64_t)sink + recent > budget || new_width < 0 || new_stride < 0)
    return KEOPS_ERR_INVALID_ARG;
  if (c->seqs > 0) {
    if (!c->weights || !kept || !new_lens || !aligned(kept, 4) || !aligned(new_lens, 4)) return KEOPS_ERR_INVALID_ARG;
    if (new_width > 0 && (!new_table || !aligned(new_table, 4))) return KEOPS_ERR_INVALID_ARG;
    // every kept slot has a place in the new table
    if (new_width < std::min<int64_t>(ceil_div(budget, c->page_size), c->table_width)) return KEOPS_ERR_INVALID_ARG;
    const int64_t kb = cut((double)c->seqs * c->heads * (double)budget * 4.0), nb = (int64_t)c->seqs * 4;
    const int64_t pb = pages_extent(*c), wb = weights_extent(*c);
    if (overlaps(kept, kb, new_lens, nb) || overlaps(kept, kb, c->lens, nb) || overlaps(new_lens, nb, c->lens, nb) ||
        overlaps(kept, kb, c->weights, wb) || overlaps(kept, kb, c->k_pages, pb) || overlaps(kept, kb, c->v_pages, pb))
      return KEOPS_ERR_INVALID_ARG;
  }
  if (!launchable(std::ceil((double)c->seqs * c->heads * (double)budget * (double)(c->dim * width_of(c->type) / 16) / 256.0), 256) ||
      (double)c->table_width * (double)c->page_size > (double)kMaxSlots ||
      !launchable((double)c->seqs * c->heads, kSelectThreads) ||
      (double)c->pages * c->heads * (double)c->page_size > 4294967295.0)       // the selection's 32-bit weight numbers
    return KEOPS_ERR_UNSUPPORTED;
  if (c->seqs == 0) return KEOPS_OK;
  (void)hipGetLastError();
  EvictArgs a{};
  a.c = view_of(*c);
  a.itemsize = (int)width_of(c->type);
  a.new_table = new_table;
  a.new_stride = new_stride;
  a.new_width = (uint32_t)new_width;
  a.budget = budget;
  a.sink = sink;
  a.recent = recent;
  a.kept = kept;
  a.new_lens = new_lens;
  launch_evict(a, st);
  return check_launch();
}

// A row in at most 64 pieces of whole steps (the pieces' sums are joined by one wave).
void plan_verify(VerifyArgs *a) {
  a->piece = (int32_t)(ceil_div(ceil_div(a->vocab, 64), kVerifyPiece) * kVerifyPiece);
  a->pieces = (int32_t)ceil_div(a->vocab, a->piece);
}

int check_verify(int seqs, int drafts, int vocab) {
  if (seqs < 0 || drafts < 0 || vocab < 1) return KEOPS_ERR_INVALID_ARG;
  if (drafts > 1 << 20 || vocab > 1 << 30) return KEOPS_ERR_UNSUPPORTED;
  VerifyArgs a{};
  a.vocab = vocab;
  plan_verify(&a);
  return launchable((double)seqs * a.pieces, kVerifyThreads) ? KEOPS_OK : KEOPS_ERR_UNSUPPORTED;
}

int verify_entry(VerifyArgs a, void *workspace, int64_t workspace_bytes, hipStream_t st) {
  if (int rc = check_verify(a.seqs, a.drafts, a.vocab)) return rc;
  for (const void *p : {(const void *)a.target, (const void *)a.draft, (const void *)a.tokens, (const void *)a.counts,
                        (const void *)a.u_accept, (const void *)a.u_sample, (const void *)a.out, (const void *)a.accepted})
    if (!aligned(p, 4)) return KEOPS_ERR_INVALID_ARG;
  if (workspace && (!aligned(workspace, 256) || workspace_bytes < 0)) return KEOPS_ERR_INVALID_ARG;
  if (a.seqs == 0) return KEOPS_OK;
  if (!a.target || !a.counts || !a.u_sample || !a.out || !a.accepted) return KEOPS_ERR_INVALID_ARG;
  if (a.drafts > 0 && (!a.tokens || !a.u_accept)) return KEOPS_ERR_INVALID_ARG;
  const int64_t ob = (int64_t)a.seqs * (a.drafts + 1) * 4, ab = (int64_t)a.seqs * 4, kb = (int64_t)a.seqs * a.drafts * 4;
  if ((double)ob * a.vocab > kMaxWorkspace) return KEOPS_ERR_UNSUPPORTED;
  const int64_t tb = ob * a.vocab, db = kb * a.vocab;
  if (overlaps(a.out, ob, a.accepted, ab)) return KEOPS_ERR_INVALID_ARG;
  const struct { const void *p; int64_t bytes; } inputs[] = {{a.target, tb}, {a.draft, db}, {a.tokens, kb}, {a.counts, ab},
                                                            {a.u_accept, kb}, {a.u_sample, ab}};
  for (const auto &in : inputs)
    if (overlaps(a.out, ob, in.p, in.bytes) || overlaps(a.accepted, ab, in.p, in.bytes)) return KEOPS_ERR_INVALID_ARG;
  (void)hipGetLastError();
  plan_verify(&a);
  Workspace own;
  char *ws = nullptr;
  if (int rc = take_workspace(own, workspace, workspace_bytes, (int64_t)a.seqs * a.pieces * 16, st, &ws)) return rc;
  a.sums = (double2 *)ws;
  launch_verify(a, st);
  return check_launch();
}

}  // namespace
}  // namespace kmi

using namespace kmi;

extern "C" {

int keops_cache_append(const keops_cache_t *cache, const void *k, const void *v, int64_t k_stride, int64_t v_stride,
                       int32_t type, const int32_t *starts, int64_t tokens, void *stream) {
  try {
    return append_entry(cache, k, v, k_stride, v_stride, type, starts, tokens, (hipStream_t)stream);
  } catch (...) {
    return KEOPS_ERR_ALLOC;
  }
}

int keops_paged_attention(const keops_cache_t *cache, const void *q, int64_t q_stride, int32_t type, int32_t heads,
                          const int32_t *starts, int64_t tokens, int32_t max_q, int32_t max_len, float scale,
                          int32_t window, float decay, void *out, float *lse, void *workspace, int64_t workspace_bytes,
                          void *stream) {
  try {
    return attend_entry(cache, q, q_stride, type, heads, starts, tokens, max_q, max_len, scale, window, decay, out, lse,
                        workspace, workspace_bytes, (hipStream_t)stream);
  } catch (...) {
    return KEOPS_ERR_ALLOC;
  }
}

int keops_paged_attention_workspace(const keops_cache_t *cache, int32_t type, int32_t heads, int64_t tokens,
                                    int32_t max_q, int32_t max_len, int32_t window, int64_t *bytes) {
  try {
    if (!bytes) return KEOPS_ERR_INVALID_ARG;
    *bytes = 0;
    if (int rc = check_attend(cache, type, tokens, heads, max_q, max_len, 1.0f, window, 0.0f)) return rc;
    if (!has_work(*cache, tokens, max_q)) return KEOPS_OK;
    int cus = 0;
    if (int rc = device_setup(&cus)) return rc;
    AttendPlan p;
    if (int rc = plan_attend(*cache, type, tokens, heads, tokens ? max_q : 0, max_len, window, cus, &p)) return rc;
    *bytes = p.total();
    return KEOPS_OK;
  } catch (...) {
    return KEOPS_ERR_ALLOC;
  }
}

int keops_cache_evict(const keops_cache_t *cache, const int32_t *new_table, int64_t new_stride, int32_t new_width,
                      int32_t budget, int32_t sink, int32_t recent, int32_t *kept, int32_t *new_lens, void *stream) {
  try {
    return evict_entry(cache, new_table, new_stride, new_width, budget, sink, recent, kept, new_lens, (hipStream_t)stream);
  } catch (...) {
    return KEOPS_ERR_ALLOC;
  }
}

int keops_verify_draft(const float *target, const float *draft, const int32_t *tokens, const int32_t *counts,
                       const float *u_accept, const float *u_sample, int32_t seqs, int32_t drafts, int32_t vocab,
                       int32_t *out, int32_t *accepted, void *workspace, int64_t workspace_bytes, void *stream) {
  try {
    VerifyArgs a{};
    a.target = target; a.draft = draft; a.tokens = tokens; a.counts = counts;
    a.u_accept = u_accept; a.u_sample = u_sample;
    a.seqs = seqs; a.drafts = drafts; a.vocab = vocab;
    a.out = out; a.accepted = accepted;
    return verify_entry(a, workspace, workspace_bytes, (hipStream_t)stream);
  } catch (...) {
    return KEOPS_ERR_ALLOC;
  }
}

int keops_verify_draft_workspace(int32_t seqs, int32_t drafts, int32_t vocab, int64_t *bytes) {
  if (!bytes) return KEOPS_ERR_INVALID_ARG;
  *bytes = 0;
  if (int rc = check_verify(seqs, drafts, vocab)) return rc;
  VerifyArgs a{};
  a.vocab = vocab;
  plan_verify(&a);
  *bytes = (int64_t)seqs * a.pieces * 16;
  return KEOPS_OK;
}

}  // extern "C"
