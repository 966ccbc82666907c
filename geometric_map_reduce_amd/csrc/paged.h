// paged.h -- internal definitions of the paged key/value cache operators: the
// launch arguments, slot addressing and the 16-bit / 8-bit element types.
#pragma once

#include "common.h"

namespace kmi {

enum CacheType : int { CT_BF16 = 0, CT_F16 = 1, CT_E4M3 = 2 };

// n / d for n < 2^31: q = (n * mul) >> shift with mul = floor(2^(31+s) / d) + 1,
// s = ceil(log2 d).  The excess of mul over the exact quotient is at most 1, so the
// product is high by at most n / 2^(31+s) < 1/d, which never reaches the next whole number.
struct FastDiv {
  uint32_t mul, shift, d;
};
inline FastDiv make_fastdiv(uint32_t d) {
  uint32_t s = 0;
  while (((uint64_t)1 << s) < d) ++s;
  return {(uint32_t)((((uint64_t)1 << (31 + s)) / d) + 1), 31 + s, d};
}
__device__ __forceinline__ uint32_t fast_div(const FastDiv &f, uint32_t n) {
  return (uint32_t)(((uint64_t)n * f.mul) >> f.shift);
}

// The cache and the batch that uses it.  Strides are in bytes.
struct CacheView {
  char *k, *v;
  float *weights;               // [pages][heads][page_size] or null
  const float *k_scale, *v_scale;
  int64_t page_stride, slot_stride, head_stride;
  FastDiv page;                 // divides a slot number by the page size
  uint32_t pages;
  int32_t heads, dim;
  const int32_t *table;         // [seqs][table_stride]
  int64_t table_stride;
  uint32_t table_width;
  const int32_t *lens;
  int32_t seqs;
};

// A slot's place: its page number and its row in it; page < 0 where the table has none
// (past its width, or an entry outside [0, pages)): such a slot is treated as absent.
struct SlotPlace {
  int32_t page;
  uint32_t row;
};
__device__ __forceinline__ SlotPlace slot_place(const CacheView &c, const int32_t *trow, uint32_t j) {
  const uint32_t pi = fast_div(c.page, j);
  int32_t pg = -1;
  if (pi < c.table_width) pg = trow[pi];
  if ((uint32_t)pg >= c.pages) pg = -1;
  return {pg, j - pi * c.page.d};
}
__device__ __forceinline__ int64_t place_offset(const CacheView &c, SlotPlace p) {
  return p.page < 0 ? -1 : (int64_t)p.page * c.page_stride + (int64_t)p.row * c.slot_stride;
}

// Slots of a sequence at most: sums of a slot, a window and a tile stay in 32 bits.
constexpr int32_t kMaxSlots = 1 << 30;

// Lane l takes lane l - N's value within its row of 16 (ROW), or lanes of later rows take an earlier row's
// last; lanes without a source take 0.  Few cycles each, where a shuffle by way of LDS takes some hundred.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xf, false);
}
// Inclusive sums over the lanes of a wave.
__device__ __forceinline__ uint32_t wave_scan_u32(uint32_t v) {
  v += dpp_u32<0x111, 0xf>(v);       // row_shr 1, 2, 4, 8
  v += dpp_u32<0x112, 0xf>(v);
  v += dpp_u32<0x114, 0xf>(v);
  v += dpp_u32<0x118, 0xf>(v);
  v += dpp_u32<0x142, 0xa>(v);       // the last of rows 0 and 2 to rows 1 and 3
  v += dpp_u32<0x143, 0xc>(v);       // the last of row 1 to rows 2 and 3
  return v;
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_f64(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, (uint64_t)dpp_u32<CTRL, ROWS>((uint32_t)b) | (uint64_t)dpp_u32<CTRL, ROWS>((uint32_t)(b >> 32)) << 32);
}
__device__ __forceinline__ double wave_scan_f64(double v) {
  v += dpp_f64<0x111, 0xf>(v);
  v += dpp_f64<0x112, 0xf>(v);
  v += dpp_f64<0x114, 0xf>(v);
  v += dpp_f64<0x118, 0xf>(v);
  v += dpp_f64<0x142, 0xa>(v);
  v += dpp_f64<0x143, 0xc>(v);
  return v;
}

// New tokens of a sequence: tokens t0 .. t0 + m of the batch, in slots first .. n of the
// sequence's n slots.  Values outside the call's bounds are cut to them.
struct SeqSpan {
  int64_t t0;
  int32_t m, n, first;
};
__device__ __forceinline__ SeqSpan seq_span(const int32_t *starts, const int32_t *lens, int s, int64_t tokens,
                                            int32_t max_q, int32_t max_len) {
  int64_t a = starts[s], b = starts[s + 1];
  a = a < 0 ? 0 : (a > tokens ? tokens : a);
  b = b < a ? a : (b > tokens ? tokens : b);
  const int32_t cnt = (int32_t)(b - a);
  int32_t n = lens[s];
  n = n < 0 ? 0 : (n > kMaxSlots ? kMaxSlots : n);
  SeqSpan r;
  r.t0 = a;
  r.first = n - cnt;
  r.m = cnt < max_q ? cnt : max_q;
  r.n = n < max_len ? n : max_len;
  return r;
}

struct AppendArgs {
  CacheView c;
  const char *k, *v;
  int64_t k_stride, v_stride;   // bytes from token to token
  const int32_t *starts;
  int64_t tokens;
};

struct AttendArgs {
  CacheView c;
  const char *q;
  int64_t q_stride;             // bytes from token to token
  const int32_t *starts;
  int64_t tokens;
  int32_t group;                // query heads that share a key/value head
  FastDiv gdiv;
  int32_t max_q, max_len, window;
  float scale_log2;             // score scale * log2(e)
  float decay;
  char *out;                    // [tokens][heads * group][dim]
  float *lse;                   // [tokens][heads * group]
  // parts of a row's sums: many rows [nsplit][tokens][heads * group], few rows [work-groups][2][rows]
  int32_t nsplit;
  uint32_t *line;               // few rows: where each sequence's tiles begin, and a work-group's share [seqs + 1]
  int32_t whole;                // few rows: a work-group has all slots of one (sequence, head); 2: of eight waves
  int32_t join_slices;          // few rows: work-groups that share the columns of a row in the join
  bool far;                     // few rows, not `whole`: the bounds allow for more keys and values than a cache holds
  float *part_o;                // [..][dim], sums under the part's maximum
  float2 *part_ml;              // (maximum in log2 units, sum)
  // few-rows form with weights: scores [seqs * heads][score_stride / 4][rows][4] in log2 units
  float *scores;
  int64_t score_stride;
  int32_t score_rows;
  // many-rows weights: partial sums [nrow][seqs * heads][max_len]
  int32_t nrow;
  float *part_w;
};

struct EvictArgs {
  CacheView c;
  int itemsize;
  const int32_t *new_table;
  int64_t new_stride;
  uint32_t new_width;
  int32_t budget, sink, recent;
  int32_t *kept, *new_lens;
};

struct VerifyArgs {
  const float *target, *draft;
  const int32_t *tokens, *counts;
  const float *u_accept, *u_sample;
  int32_t seqs, drafts, vocab;
  int32_t *out, *accepted;
  int32_t pieces, piece;        // a row's pieces (at most 64) and the indices of one
  double2 *sums;                // [seqs][pieces]: what is left of the target's row, and all of it
};
constexpr int kVerifyPiece = 2048;   // indices that a work-group takes at a time

// ---------------------------------------------------------------- launches
void launch_append(const AppendArgs &a, int type, int cache_type, hipStream_t st);
// Variants exist for dim 64, 96, 128 and 256; the API checks before it calls.
constexpr int kFewRowsMax = 32;      // rows (new tokens x group) of the few-rows form
constexpr int kManyRowsTile = 128;   // rows of a work-group of the many-rows form
constexpr int kSumSlotsTile = 256;   // slots of a work-group of the column sums
// Threads of a work-group, for the plans.
constexpr int kFinishThreads = 256;  // few rows: the second pass
constexpr int kJoinThreads = 256;    // many rows: the join
constexpr int kSelectThreads = 1024; // eviction: the selection
constexpr int kVerifyThreads = 256;
constexpr int kScoreSlots = 2048;    // slots of a work-group that turns kept scores into weights
// Groups of threads that share a row of the many-rows join, and its work-groups.
inline int join_per_row(int dim, int nsplit) {
  const int groups = kJoinThreads / (dim / 4);
  return nsplit <= 4 ? 1 : (nsplit < groups ? nsplit / 4 : groups);
}
inline int64_t join_blocks(int64_t rows, int dim, int nsplit) {
  const int64_t rows_per = kJoinThreads / (dim / 4) / join_per_row(dim, nsplit);
  return (rows + rows_per - 1) / rows_per;
}
// Both passes.  grid 0: the work-groups of the variant that a compute unit holds (-1: HIP error).
// join_rows: rows of a work-group that joins parts, 0: there are none.
int launch_attend_few(const AttendArgs &a, int type, bool e4m3, int dim, int row_tiles, int grid, int join_rows,
                      hipStream_t st);
void launch_attend_many(const AttendArgs &a, int type, bool e4m3, int dim, dim3 grid, hipStream_t st);
void launch_attend_sums(const AttendArgs &a, int type, bool e4m3, int dim, dim3 grid, hipStream_t st);
void launch_attend_join(const AttendArgs &a, int type, hipStream_t st);
void launch_attend_sums_join(const AttendArgs &a, hipStream_t st);
void launch_evict(const EvictArgs &a, hipStream_t st);
void launch_verify(const VerifyArgs &a, hipStream_t st);

// ---------------------------------------------------------------- element types
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short s16x2 __attribute__((ext_vector_type(2)));

// kShift: p is computed 2^kShift larger.  fp16 ends at 2^-24, and 10^5 slots below that would add up
// to some 10^-3 of a sum; with p up to 2^15 (2^8 by the lazy maximum, 2^7 here) it ends at 2^-31 of the
// largest.
struct Bf16 {
  static constexpr float kShift = 0.0f;
  static constexpr uint32_t kExp = 0x7f807f80u;   // exponent bits of a pair
  static __device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
  // two floats to a pair, to nearest even
  static __device__ __forceinline__ uint32_t pack(float x, float y) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){x, y}, bf16x2));
  }
  static __device__ __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
  static __device__ __forceinline__ float hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
  // two of four e4m3 values to a pair (exact)
  template <bool HI>
  static __device__ __forceinline__ uint32_t from_e4m3(uint32_t w) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HI));
  }
};
struct F16 {
  static constexpr float kShift = 7.0f;
  static constexpr uint32_t kExp = 0x7c007c00u;
  static __device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ uint32_t pack(float x, float y) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){x, y}, f16x2));
  }
  static __device__ __forceinline__ float lo(uint32_t w) { return (float)__builtin_bit_cast(f16x2, w).x; }
  static __device__ __forceinline__ float hi(uint32_t w) { return (float)__builtin_bit_cast(f16x2, w).y; }
  template <bool HI>
  static __device__ __forceinline__ uint32_t from_e4m3(uint32_t w) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, HI));
  }
};

// A half of w where it is an infinity or a NaN, 0 where it is finite.
template <class T>
__device__ __forceinline__ float nonfinite_lo(uint32_t w) {
  return (w & T::kExp & 0xffffu) == (T::kExp & 0xffffu) ? T::lo(w) : 0.0f;
}
template <class T>
__device__ __forceinline__ float nonfinite_hi(uint32_t w) {
  return (w & T::kExp & 0xffff0000u) == (T::kExp & 0xffff0000u) ? T::hi(w) : 0.0f;
}
// Zeros for the halves of w that are infinities or NaNs.
template <class T>
__device__ __forceinline__ uint32_t finite_halves(uint32_t w) {
  const uint32_t lo = (w & T::kExp & 0xffffu) == (T::kExp & 0xffffu) ? 0xffffu : 0u;
  const uint32_t hi = (w & T::kExp & 0xffff0000u) == (T::kExp & 0xffff0000u) ? 0xffff0000u : 0u;
  return w & ~(lo | hi);
}
// Zeros for the bytes of w that are NaNs as e4m3.
__device__ __forceinline__ uint32_t finite_bytes(uint32_t w) {
  const uint32_t t = (w & 0x7f7f7f7fu) ^ 0x7f7f7f7fu;                // 0 where the byte is a NaN
  const uint32_t nan = (~(t + 0x7f7f7f7fu) & 0x80808080u) >> 7;      // no carry passes a byte
  return w & ~(nan * 255u);
}
// The lowest n of 32 bits; none for n <= 0.
__device__ __forceinline__ uint32_t first_bits(int n) {
  return n <= 0 ? 0u : (n >= 32 ? 0xffffffffu : (1u << n) - 1u);
}
template <class T>
__device__ __forceinline__ bool clear_nonfinite(u32x4 &x) {
  bool any = false;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const uint32_t y = finite_halves<T>(x[u]);
    any |= y != x[u];
    x[u] = y;
  }
  return any;
}

template <class T>
__device__ __forceinline__ u32x4 widen_e4m3(u32x2 w) {
  return (u32x4){T::template from_e4m3<false>(w.x), T::template from_e4m3<true>(w.x),
                 T::template from_e4m3<false>(w.y), T::template from_e4m3<true>(w.y)};
}

// A load of what is read once, past the caches if FAR.
template <class V, bool FAR>
__device__ __forceinline__ V load_once(const void *p) {
  return FAR ? __builtin_nontemporal_load((const V *)p) : *(const V *)p;
}
constexpr double kLastLevel = 256e6;     // bytes of the last-level cache

// Zeros where `keep` is false.
__device__ __forceinline__ u32x4 keep_if(u32x4 v, bool keep) {
  const uint32_t m = keep ? 0xffffffffu : 0u;
  return v & (u32x4){m, m, m, m};
}

}  // namespace kmi
