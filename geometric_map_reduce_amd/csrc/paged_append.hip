// paged_append.hip -- new keys and values into their slots of a paged cache.
//
//   pages[table[s, j / page]][j % page][h] = k[t, h]      j = first_s + (t - starts_s)
//
// for every token t of every sequence s (8-bit caches: the e4m3 value nearest to
// k / k_scale[h], cut to +-448; 4-bit ones: blocks of 32 columns, four threads each, under a power of two
// that their largest magnitude decides), and weight 0 for the slot where weights are kept.  A copy:
// each element is read once and written once, so memory bounds a long prompt (16,384 tokens of 8 x 128
// bf16 with weights: 28 us a call, 4.8 TB/s, the rate of a large copy) and a chain of loads a single
// step: the halving of starts, its own start and length, the table's entry (64 sequences: nine loads in turn, 3.5 us
// of the GPU's time with the launch).
#include "step.h"

namespace kmi {
namespace {

constexpr int kAppendThreads = 256;

template <bool BF>
__device__ __forceinline__ float widen16(uint32_t w, int hi) {
  const uint16_t b = hi ? (uint16_t)(w >> 16) : (uint16_t)w;
  if (BF) return __uint_as_float((uint32_t)b << 16);
  return (float)__builtin_bit_cast(_Float16, b);
}

// One thread moves 8 elements (16 bytes) of a key row and the same 8 of the value row.
// Threads of a token are adjacent, so its row of heads x dim elements is read in one
// sweep; each thread finds the owner sequence in the sorted starts by halving.
template <bool BF, int BITS>
__global__ __launch_bounds__(kAppendThreads) void append_kernel(AppendArgs a) {
  constexpr bool E4M3 = BITS == 8, E2M1 = BITS == 4;
  const int per = a.c.heads * a.c.dim / 8;   // 8-element pieces of a token
  const int64_t piece = (int64_t)blockIdx.x * kAppendThreads + threadIdx.x;
  const int64_t t = piece / per;
  const int e = (int)(piece - t * per);
  const bool live = t < a.tokens;
  // last s with starts[s] <= t (the wave's lanes may hold different tokens)
  int lo = 0, hi = a.c.seqs;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.starts[mid] <= t) lo = mid; else hi = mid;
  }
  if (!live) return;
  // the slot that attention takes the token to be in, starts outside the tokens included
  const SeqSpan sp = seq_span(a.starts, a.c.lens, lo, a.tokens, 0x7fffffff, 0x7fffffff);
  if (t < sp.t0 || t >= sp.t0 + sp.m) return;
  const int64_t j = sp.first + (t - sp.t0);
  if (j < 0) return;
  const SlotPlace p = slot_place(a.c, a.c.table + (int64_t)lo * a.c.table_stride, (uint32_t)j);
  if (p.page < 0) return;
  const int h = e * 8 / a.c.dim, d = e * 8 - h * a.c.dim;
  const u32x4 kv = *(const u32x4 *)(a.k + t * a.k_stride + (int64_t)e * 16);
  const u32x4 vv = *(const u32x4 *)(a.v + t * a.v_stride + (int64_t)e * 16);
  const int64_t off = place_offset(a.c, p) + (int64_t)h * a.c.head_stride + (int64_t)d * BITS / 8;
  if (E2M1) {
    using T = typename std::conditional<BF, Bf16, F16>::type;
    float x[8], y[8];
    widen8<T>(kv, x);
    widen8<T>(vv, y);
    uint32_t kp, vp;
    *(uint32_t *)(a.c.k + off) = to_e2m1(x, T::kE2m1Top, &kp);
    *(uint32_t *)(a.c.v + off) = to_e2m1(y, T::kE2m1Top, &vp);
    if (d % kPowerBlock == 0) {
      const uint64_t at = (uint64_t)place_number(a.c, p, h) * (a.c.dim / kPowerBlock) + d / kPowerBlock;
      a.c.k_power[at] = (uint8_t)kp;
      a.c.v_power[at] = (uint8_t)vp;
    }
  } else if (E4M3) {
    const float ks = a.c.k_scale[h], vs = a.c.v_scale[h];
    u32x2 ko, vo;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      int pk = 0, pv = 0;
      pk = __builtin_amdgcn_cvt_pk_fp8_f32(e4m3_quotient(widen16<BF>(kv[2 * w], 0), ks),
                                           e4m3_quotient(widen16<BF>(kv[2 * w], 1), ks), pk, false);
      pk = __builtin_amdgcn_cvt_pk_fp8_f32(e4m3_quotient(widen16<BF>(kv[2 * w + 1], 0), ks),
                                           e4m3_quotient(widen16<BF>(kv[2 * w + 1], 1), ks), pk, true);
      pv = __builtin_amdgcn_cvt_pk_fp8_f32(e4m3_quotient(widen16<BF>(vv[2 * w], 0), vs),
                                           e4m3_quotient(widen16<BF>(vv[2 * w], 1), vs), pv, false);
      pv = __builtin_amdgcn_cvt_pk_fp8_f32(e4m3_quotient(widen16<BF>(vv[2 * w + 1], 0), vs),
                                           e4m3_quotient(widen16<BF>(vv[2 * w + 1], 1), vs), pv, true);
      ko[w] = (uint32_t)pk;
      vo[w] = (uint32_t)pv;
    }
    *(u32x2 *)(a.c.k + off) = ko;
    *(u32x2 *)(a.c.v + off) = vo;
  } else {
    *(u32x4 *)(a.c.k + off) = kv;
    *(u32x4 *)(a.c.v + off) = vv;
  }
  if (a.c.weights && d == 0)
    a.c.weights[((int64_t)p.page * a.c.heads + h) * a.c.page.d + p.row] = 0.0f;
}

}  // namespace

void launch_append(const AppendArgs &a, int type, int cache_type, hipStream_t st) {
  const int64_t pieces = a.tokens * (a.c.heads * a.c.dim / 8);
  const dim3 grid((unsigned)((pieces + kAppendThreads - 1) / kAppendThreads));
  if (cache_type == CT_E2M1) {
    if (type == CT_BF16) append_kernel<true, 4><<<grid, kAppendThreads, 0, st>>>(a);
    else append_kernel<false, 4><<<grid, kAppendThreads, 0, st>>>(a);
  } else if (cache_type == CT_E4M3) {
    if (type == CT_BF16) append_kernel<true, 8><<<grid, kAppendThreads, 0, st>>>(a);
    else append_kernel<false, 8><<<grid, kAppendThreads, 0, st>>>(a);
  } else {
    append_kernel<true, 16><<<grid, kAppendThreads, 0, st>>>(a);
  }
}

}  // namespace kmi
