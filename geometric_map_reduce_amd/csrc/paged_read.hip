// paged_read.hip -- the values in slots of a paged cache, as 16-bit rows.
//
//   k[t, h] = pages[table[s, j / page]][j % page][h],   j the slot of token t of sequence s
//
// e4m3 times its head's scale, e2m1 times its block's power of two, rounded once to the 16-bit type; 0 where the
// slot is absent.  The append's way backwards: one thread has eight columns of a key and of a value, and memory bounds it
// (16,576 slots of 8 x 128, 4 bits: 85 MB read and written in 21 us).  For prompts over a 4-bit cache the slots go the
// same way to pages of 16 bits, once, instead of in every work-group of attention.
#include "step.h"

namespace kmi {
namespace {

constexpr int kReadThreads = 256;

template <class T, int BITS>
__device__ __forceinline__ u32x4 held8(const char *at, float scale, const uint8_t *power) {
  if (BITS == 16) return *(const u32x4 *)at;
  if (BITS == 4) return widen_e2m1<T>(*(const uint32_t *)at, *power);
  const u32x2 w = *(const u32x2 *)at;
  // the product has up to 28 bits: 32 bits with an odd last place where it is not one of theirs
  const double by = (double)scale;
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], true);
    r[2 * i] = T::pack(round_to_odd(a.x * by), round_to_odd(a.y * by));
    r[2 * i + 1] = T::pack(round_to_odd(b.x * by), round_to_odd(b.y * by));
  }
  return r;
}

template <class T, int BITS>
__global__ __launch_bounds__(kReadThreads) void read_kernel(ReadArgs a) {
  const int per = a.c.heads * a.c.dim / 8;   // 8-element pieces of a token
  const int64_t piece = (int64_t)blockIdx.x * kReadThreads + threadIdx.x;
  const int64_t t = piece / per;
  const int e = (int)(piece - t * per);
  if (t >= a.tokens) return;
  int lo = 0, hi = a.c.seqs;                 // last s with starts[s] <= t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.starts[mid] <= t) lo = mid; else hi = mid;
  }
  const SeqSpan sp = seq_span(a.starts, a.c.lens, lo, a.tokens, 0x7fffffff, 0x7fffffff);
  if (t < sp.t0 || t >= sp.t0 + sp.m) return;
  const int64_t j = sp.first + (t - sp.t0);
  SlotPlace p{-1, 0};
  if (j >= 0) p = slot_place(a.c, a.c.table + (int64_t)lo * a.c.table_stride, (uint32_t)j);
  u32x4 k = (u32x4){0, 0, 0, 0}, v = k;
  if (p.page >= 0) {
    const int h = e * 8 / a.c.dim, d = e * 8 - h * a.c.dim;
    const int64_t off = place_offset(a.c, p) + (int64_t)h * a.c.head_stride + d * BITS / 8;
    const uint64_t at = BITS == 4 ? (uint64_t)place_number(a.c, p, h) * (a.c.dim / kPowerBlock) + d / kPowerBlock : 0;
    k = held8<T, BITS>(a.c.k + off, BITS == 8 ? a.c.k_scale[h] : 1.0f, a.c.k_power + at);
    v = held8<T, BITS>(a.c.v + off, BITS == 8 ? a.c.v_scale[h] : 1.0f, a.c.v_power + at);
  }
  *(u32x4 *)(a.k + t * a.k_stride + (int64_t)e * 16) = k;
  *(u32x4 *)(a.v + t * a.v_stride + (int64_t)e * 16) = v;
}

// A thread has eight columns of a slot's key and value, as above; the slots that no row sees are left out.
template <class T>
__global__ __launch_bounds__(kReadThreads) void widen_kernel(WidenArgs a) {
  const uint32_t per = (uint32_t)(a.c.heads * a.c.dim / 8), ps = a.c.page.d;
  const int64_t id = (int64_t)blockIdx.x * kReadThreads + threadIdx.x;
  const int64_t at = id / per;                       // the slot, of all that the new pages have
  const uint32_t e = (uint32_t)(id - at * per);
  const int64_t slots = (int64_t)a.width * ps;
  const int s = (int)(at / slots);
  if (s >= a.c.seqs) return;
  const uint32_t j = (uint32_t)(at - (int64_t)s * slots);
  const SlotPlace p = slot_place(a.c, a.c.table + (int64_t)s * a.c.table_stride, j);
  const uint32_t pi = fast_div(a.c.page, j), to = (uint32_t)s * (uint32_t)a.width + pi;
  if (e == 0 && p.row == 0) a.table[to] = p.page < 0 ? -1 : (int32_t)to;
  const SeqSpan sp = seq_span(a.starts, a.c.lens, s, a.tokens, a.max_q, a.max_len);
  // from the start of the first tile of attention that has a slot that some row sees: what was left in the others
  // by an earlier call, infinities and NaN among it, would have to be cleared from the tile (81 us with a window, 154 so)
  int from = a.window > 0 ? sp.first - a.window + 1 : 0;
  from = from > 0 ? from / kManySlotsTile * kManySlotsTile : 0;
  if (p.page < 0 || (int)j >= sp.n || (int)j < from || sp.m == 0) return;
  const int h = (int)(e * 8 / a.c.dim), d = (int)(e * 8) - h * a.c.dim;
  const int64_t off = place_offset(a.c, p) + (int64_t)h * a.c.head_stride + d / 2;
  const uint64_t power = (uint64_t)place_number(a.c, p, h) * (a.c.dim / kPowerBlock) + d / kPowerBlock;
  const u32x4 k = widen_e2m1<T>(*(const uint32_t *)(a.c.k + off), a.c.k_power[power]);
  const u32x4 v = widen_e2m1<T>(*(const uint32_t *)(a.c.v + off), a.c.v_power[power]);
  // [page][head][row][dim]
  const int64_t out = ((((int64_t)to * a.c.heads + h) * ps + p.row) * a.c.dim + d) * 2;
  *(u32x4 *)(a.k + out) = k;
  *(u32x4 *)(a.v + out) = v;
}

}  // namespace

void launch_widen(const WidenArgs &a, int type, hipStream_t st) {
  const int64_t pieces = (int64_t)a.c.seqs * a.width * a.c.page.d * (a.c.heads * a.c.dim / 8);
  const dim3 grid((unsigned)((pieces + kReadThreads - 1) / kReadThreads));
  if (type == CT_BF16) widen_kernel<Bf16><<<grid, kReadThreads, 0, st>>>(a);
  else widen_kernel<F16><<<grid, kReadThreads, 0, st>>>(a);
}

void launch_read(const ReadArgs &a, int type, int bits, hipStream_t st) {
  const int64_t pieces = a.tokens * (a.c.heads * a.c.dim / 8);
  const dim3 grid((unsigned)((pieces + kReadThreads - 1) / kReadThreads));
  if (bits == 16) {
    read_kernel<Bf16, 16><<<grid, kReadThreads, 0, st>>>(a);
  } else if (bits == 8) {
    if (type == CT_BF16) read_kernel<Bf16, 8><<<grid, kReadThreads, 0, st>>>(a);
    else read_kernel<F16, 8><<<grid, kReadThreads, 0, st>>>(a);
  } else {
    if (type == CT_BF16) read_kernel<Bf16, 4><<<grid, kReadThreads, 0, st>>>(a);
    else read_kernel<F16, 4><<<grid, kReadThreads, 0, st>>>(a);
  }
}

}  // namespace kmi
