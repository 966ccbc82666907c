// paged_many.h -- attention of many rows over a paged cache (a prompt, or a chunk of one), and
// the column sums that give every slot the attention it received.
//
//   out[t, g] = sum_j p_j v_j,   p_j = exp(z_j - lse),  z_j = scale <q[t, g], k_j>
//   w[j]      = sum over the rows (t, g) of a key/value head of p_j
//
// Attention: a work-group takes 128 rows of one (sequence, key/value head), 32 a wave, and walks
// the slots that any of them sees in tiles of 64.  Tiles of K and V lie in LDS, the next ones on
// their way while one is used.  The matrix products and the clock that they leave bound it: 4,096
// tokens after 12,288 slots (32/8 heads of 128, bf16) take 946 to 967 us, by card, 1,017 TFLOP/s where a
// large library product reaches 1,268 (1,120 us on a card that runs that at 1,199).
//
//  * S^T = K Q^T with 32 x 32 x 16 products: Q stays in registers as the B operand, a lane holds one row
//    and 16 slots of each 32.  Counting the slots in that order makes the packed p the B operand
//    of O^T = V^T P^T as it stands, and V^T is read from the row-major tile with transposing
//    LDS reads.
//  * Which slots a row sees are bits: the slots that are there, the slot of the token, the window.  Only
//    tiles where some row does not see some slot look at them.
//  * Running maximum, sums, absent slots, non-finite values and the rounding of p to 16 bits for the
//    matrix product as in the few-rows form.
//  * 4-bit caches: from 1,024 rows of a head on the slots are widened to 16 bits once, before (paged_read.hip), since
//    each of the many work-groups of a head would do it again; fewer rows widen their tiles on the way to LDS.
//  * Few rows and long caches: the slots are split over as many work-groups as the device holds at
//    once, and a second kernel joins the parts.
//
// Column sums: one pass over Q with K in registers.  The rows' lse is known, so
// p = exp(z - lse) needs no running maximum; a wave owns 64 slots and adds up the rows of Q tiles
// staged in LDS.  Nine prompts of up to 777 tokens with a window of 1,024 (16/4 heads of 64) take 34 us.
// Waiting bounds that: matrix instructions take 3 us of it and vector instructions, the exponentials among
// them, 8, and the waves stand still for 44 % of their time (counters): 3,600 short work-groups, each with a
// chain length, table, key before its first product and a barrier a tile.  A tile's arithmetic has no branch:
// hidden slots get a score of -inf by selection (left to a condition each, 64 jumps a tile, it took 45 us).
#pragma once

#include <type_traits>

#include "paged.h"

namespace kmi {

constexpr int kManyThreads = 256;
constexpr float kManyLazy = 8.0f;   // log2 of what a score may pass the running maximum by

typedef short s16x4 __attribute__((ext_vector_type(4)));

// Piece (16 bytes) p of row r of a tile with D 16-bit columns lies at piece p ^ x(r).  A read of a wave
// goes in parts of 256 bytes over 64 banks: 16 rows' pieces of K (rows 0-3, 12-15, 20-23, 24-27 and so
// on), 4 rows' quadruples of V.  With these x no two of a part share a bank (counted: none; with a
// rotation by 8 pieces instead of 16 half of the LDS cycles at D = 128 were conflicts).
template <int D>
__device__ __forceinline__ int k_swizzle(int r) { return D == 96 ? (r >> 2) & 3 : (D == 64 ? (r >> 1) & 7 : r & 15); }
template <int D>
__device__ __forceinline__ int v_swizzle(int r) { return D == 96 ? 0 : (D == 64 ? 2 * (r & 3) : 4 * (r & 3)); }

__device__ __forceinline__ float half_max(float v) { return fmaxf(v, __shfl_xor(v, 32)); }
__device__ __forceinline__ float half_sum(float v) { return v + __shfl_xor(v, 32); }

// Slot of accumulator register r in a 32-slot tile for a lane of half hi.
__device__ __forceinline__ constexpr int slot32(int r, int hi) { return hi * 4 + (r & 3) + 8 * (r >> 2); }

// 16 bytes a lane from global memory to LDS, lane l's at lds + 16 l, without passing registers.
// Done when vmcnt says so: the compiler does not know, dma_wait() does.  (M0 needs one wait state.)  M0 is named
// as changed: the compiler keeps no value in it for long, and warns of that, but may set it once for two of its
// own uses that this lies between.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void dma16(const void *from, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(from) : "memory", "m0");
}
#pragma clang diagnostic pop
template <int LEFT>
__device__ __forceinline__ void dma_wait() { asm volatile("s_waitcnt vmcnt(%0)" ::"n"(LEFT) : "memory"); }
__device__ __forceinline__ uint32_t lds_address(const void *p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const char *)p;
}

template <class T, int BITS, int D>
__global__ __launch_bounds__(kManyThreads, D > 128 ? 1 : 2) void attend_many_kernel(AttendArgs a) {
  constexpr bool E4M3 = BITS == 8, E2M1 = BITS == 4, NARROW = E4M3 || E2M1;
  // slots of a tile: two halves are two independent chains of products (one of 32 waited for itself:
  // D = 256 ran at 647 instead of 759 TFLOP/s)
  constexpr int KT = kManySlotsTile;
  constexpr int kSteps = D / 16, kCols = D / 32, kSub = KT / 32;
  constexpr int kPieces = D / 8;                     // 16-byte pieces of a row in LDS
  constexpr int kLoads = KT * kPieces / kManyThreads;
  // tiles in LDS: as many as leave room for two work-groups on a compute unit (one at D = 256; 8-bit
  // and 4-bit ones pass registers, one ahead)
  constexpr int kBufs = NARROW ? 2 : (D == 64 ? 4 : (D == 96 ? 3 : 2));
  constexpr int kChunk = D == 96 ? 4 : 8;            // tiles whose addresses are placed together
  constexpr int kPlace = kChunk * KT / kManyThreads; // slots a thread places
  static_assert(kBufs <= kChunk, "a chunk is placed before the first fetch from it");
  static_assert(KT == kWave, "a wave's ballot is a tile");
  static_assert(KT * kPieces % kManyThreads == 0 && kChunk * KT % kManyThreads == 0, "whole pieces per thread");
  __shared__ __align__(16) uint16_t sk[kBufs][KT * D];
  __shared__ __align__(16) uint16_t sv[kBufs][KT * D];
  __shared__ int64_t off[2][kChunk * KT];
  __shared__ uint32_t number[E2M1 ? 2 : 1][E2M1 ? kChunk * KT : 1];     // the slots' among all powers
  __shared__ uint64_t present[2][kChunk];              // which of a tile's slots are there
  __shared__ int sh_odd;                               // a wave cleared non-finite values for all

  const int H = a.c.heads, G = a.group;
  const int64_t heads = (int64_t)H * G;
  const int rows_most = a.max_q * G;
  const int nrt = (rows_most + kManyRowsTile - 1) / kManyRowsTile;
  int b = blockIdx.x;
  const int h = b % H;
  b /= H;
  const int split = b % a.nsplit;
  b /= a.nsplit;
  const int rt = nrt - 1 - b % nrt, s = b / nrt;     // the rows that see most come first
  const int tid = threadIdx.x, lane = tid & 63, col = lane & 31, hi = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

  const SeqSpan sp = seq_span(a.starts, a.c.lens, s, a.tokens, a.max_q, a.max_len);
  const int R = sp.m * G, row0 = rt * kManyRowsTile;
  if (row0 >= R) return;
  const int rows = R - row0 < kManyRowsTile ? R - row0 : kManyRowsTile;
  // slots that any row of the tile sees
  const int tok0 = (int)fast_div(a.gdiv, (uint32_t)row0), tok1 = (int)fast_div(a.gdiv, (uint32_t)(row0 + rows - 1));
  const int first_pos = sp.first + tok0, last_pos = sp.first + tok1;
  int lo = 0;
  if (a.window > 0 && first_pos - a.window + 1 > 0) lo = first_pos - a.window + 1;
  const int end = sp.n < last_pos + 1 ? sp.n : last_pos + 1;
  lo = lo / KT * KT;
  const int all = end > lo ? (end - lo + KT - 1) / KT : 0;
  const int per = (all + a.nsplit - 1) / a.nsplit;
  const int tile0 = split * per < all ? split * per : all;
  const int tiles = tile0 + per < all ? per : all - tile0;
  lo += tile0 * KT;                                  // this split's tiles: 0 .. tiles

  const int r = row0 + wave * 32 + col;
  const int tok = (int)fast_div(a.gdiv, (uint32_t)r), g = r - tok * G;
  const bool real = r < R;
  const int pos = real ? sp.first + tok : -1;
  // a wave without rows only fetches (at D = 256 the branch costs registers: 4,096 tokens after 12,288, 32/8 heads: 2,665 us with it, 2,331 without)
  const bool idle = D <= 128 && row0 + wave * 32 >= R;
  // scores are compared before they are scaled: a negative factor's sign goes to Q, a zero one's
  // scores are zeros
  const float c0 = E4M3 ? a.scale_log2 * a.c.k_scale[h] : a.scale_log2;
  const float c = c0 == 0.0f ? 1.0f : fabsf(c0);
  const uint32_t flip = c0 < 0.0f ? 0x80008000u : 0u, keep = c0 == 0.0f ? 0u : 0xffffffffu;
  u32x4 qf[kSteps];
  {
    const char *qp = a.q + (sp.t0 + tok) * a.q_stride + ((int64_t)(h * G + g) * D + hi * 8) * 2;
#pragma unroll
    for (int st = 0; st < kSteps; ++st) {
      qf[st] = real ? *(const u32x4 *)(qp + st * 32) : (u32x4){0, 0, 0, 0};
#pragma unroll
      for (int u = 0; u < 4; ++u) qf[st][u] = (qf[st][u] ^ flip) & keep;
    }
  }
  float m_run = -INFINITY, l_run = 0.0f;             // 2^m_run is the unit of the sums
  f32x16 acc[kCols];
#pragma unroll
  for (int t = 0; t < kCols; ++t)
#pragma unroll
    for (int u = 0; u < 16; ++u) acc[t][u] = 0.0f;
  const char *kbase = a.c.k + (int64_t)h * a.c.head_stride;
  const char *vbase = a.c.v + (int64_t)h * a.c.head_stride;
  const int32_t *trow = a.c.table + (int64_t)s * a.c.table_stride;

  // Addresses of eight tiles' slots at a time: page numbers are loaded a chunk ahead of their use.
  int32_t page[kPlace];
  const auto page_load = [&](int chunk) {
#pragma unroll
    for (int i = 0; i < kPlace; ++i) {
      const int j = lo + chunk * kChunk * KT + i * kManyThreads + tid;
      page[i] = -1;
      if (j < end) page[i] = slot_place(a.c, trow, (uint32_t)j).page;
    }
  };
  const auto page_put = [&](int chunk) {
#pragma unroll
    for (int i = 0; i < kPlace; ++i) {
      const int at = i * kManyThreads + tid, j = lo + chunk * kChunk * KT + at;
      const uint32_t row = (uint32_t)j - fast_div(a.c.page, (uint32_t)j) * a.c.page.d;
      const int64_t o = place_offset(a.c, SlotPlace{page[i], row});
      off[chunk & 1][at] = NARROW || o >= 0 ? o : 0;
      if (E2M1) number[chunk & 1][at] = place_number(a.c, SlotPlace{page[i], row}, h);
      const uint64_t there = __ballot(page[i] >= 0);
      if (lane == 0) present[chunk & 1][i * 4 + wave] = there;
    }
  };
  const auto off_at = [&](int tile) -> const int64_t * { return &off[(tile / kChunk) & 1][tile % kChunk * KT]; };

  const auto there_at = [&](int tile) { return present[(tile / kChunk) & 1][tile % kChunk]; };

  // A tile on its way: 16-bit caches go straight to LDS, narrower ones by way of registers.  A thread of a 4-bit
  // one has whole blocks, 16 bytes and their power: those of K first, then those of V (no wave has both but at D = 96).
  constexpr int kBlocks = D / kPowerBlock, kItems = (2 * KT * kBlocks + kManyThreads - 1) / kManyThreads;
  uint32_t gk[E4M3 ? kLoads : 1][2], gv[E4M3 ? kLoads : 1][2];
  u32x4 gb[E2M1 ? kItems : 1];
  uint32_t gp[E2M1 ? kItems : 1];
  uint32_t held = 0;
  const auto fetch = [&](int tile) {
    const int64_t *po = off_at(tile);
    if constexpr (E2M1) {
      held = 0;
#pragma unroll
      for (int i = 0; i < kItems; ++i) {
        int id = tid + i * kManyThreads;
        const bool v = id >= KT * kBlocks;
        id -= v ? KT * kBlocks : 0;
        if (id >= KT * kBlocks) break;               // D = 96: the last half round
        const int row = id / kBlocks, b = id - row * kBlocks;
        int64_t o = po[row];
        if (o >= 0) held |= 1u << i;
        o = o < 0 ? 0 : o;
        gb[i] = *(const u32x4 *)((v ? vbase : kbase) + o + b * 16);
        gp[i] = (v ? a.c.v_power : a.c.k_power)[(uint64_t)number[(tile / kChunk) & 1][tile % kChunk * KT + row] * kBlocks + b];
      }
    } else if constexpr (E4M3) {
      held = 0;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int id = tid + i * kManyThreads, row = id / kPieces, p = id - row * kPieces;
        int64_t o = po[row];
        if (o >= 0) held |= 1u << i;
        o = o < 0 ? 0 : o;
        const u32x2 x = *(const u32x2 *)(kbase + o + p * 8);
        const u32x2 y = *(const u32x2 *)(vbase + o + p * 8);
        gk[i][0] = x.x; gk[i][1] = x.y;
        gv[i][0] = y.x; gv[i][1] = y.y;
      }
    } else {
      // an absent slot's row is some row of the pool: no row sees its K, and its V is cleared before use
      const uint32_t ldk = lds_address(sk[tile % kBufs]) + wave * 1024, ldv = lds_address(sv[tile % kBufs]) + wave * 1024;
      int64_t o[kLoads];
#pragma unroll
      for (int i = 0; i < kLoads; ++i) o[i] = po[(tid + i * kManyThreads) / kPieces];
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int id = tid + i * kManyThreads, row = id / kPieces, p = id - row * kPieces;
        dma16(kbase + (p ^ k_swizzle<D>(row)) * 16 + o[i], ldk + i * (kManyThreads * 16));
        dma16(vbase + (p ^ v_swizzle<D>(row)) * 16 + o[i], ldv + i * (kManyThreads * 16));
      }
    }
  };
  const auto arrive = [&](int tile) {
    if constexpr (E2M1) {
#pragma unroll
      for (int i = 0; i < kItems; ++i) {
        int id = tid + i * kManyThreads;
        const bool v = id >= KT * kBlocks;
        id -= v ? KT * kBlocks : 0;
        if (id >= KT * kBlocks) break;
        const int row = id / kBlocks, b = id - row * kBlocks;
        uint16_t *to = (v ? sv[tile % kBufs] : sk[tile % kBufs]) + row * D;
        const int x = v ? v_swizzle<D>(row) : k_swizzle<D>(row);
#pragma unroll
        for (int u = 0; u < 4; ++u)
          *(u32x4 *)&to[((4 * b + u) ^ x) * 8] = keep_if(widen_e2m1<T>(gb[i][u], gp[i]), (held >> i) & 1u);
      }
    } else if constexpr (E4M3) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int id = tid + i * kManyThreads, row = id / kPieces, p = id - row * kPieces;
        const u32x4 x = widen_e4m3<T>((u32x2){gk[i][0], gk[i][1]});
        const u32x4 y = widen_e4m3<T>((u32x2){gv[i][0], gv[i][1]});
        *(u32x4 *)&sk[tile % kBufs][row * D + (p ^ k_swizzle<D>(row)) * 8] = x;
        *(u32x4 *)&sv[tile % kBufs][row * D + (p ^ v_swizzle<D>(row)) * 8] = keep_if(y, (held >> i) & 1u);
      }
    } else if (tile + kBufs - 2 < tiles) {
      dma_wait<(kBufs - 2) * 2 * kLoads>();        // the tiles after this one may be on their way
    } else {
      dma_wait<0>();
    }
  };

  // In a tile with slots that some row does not see: V of absent ones is cleared, and non-finite values of
  // those that some rows see and others do not wait for the end.  Each thread looks at its own pieces.
  const auto clear = [&](int buf, int tile, uint64_t there) {
    // unrolled it takes 39 registers more at D = 96: 773 to 811 us for 4,096 tokens after 12,288; elsewhere rolled
    // is slower by a percent
    constexpr int kUnroll = D == 96 ? 1 : kLoads;
    bool odd = false;
#pragma unroll kUnroll
    for (int i = 0; i < kLoads; ++i) {
      const int id = tid + i * kManyThreads, u = id / kPieces, j = lo + tile * KT + u;
      u32x4 x = ((const u32x4 *)sv[buf])[id];
      const bool here = (there >> u) & 1u, some = j > first_pos || (a.window > 0 && j <= last_pos - a.window);
      bool change = !here;
      if (here && some && clear_nonfinite<T>(x)) odd = change = true;
      if (change) ((u32x4 *)sv[buf])[id] = keep_if(x, here);
    }
    if (odd) sh_odd = 1;
  };
  // One tile.  masked: some row may not see some slot of it.
  const auto step = [&](bool masked, int buf, int tile, uint64_t there) {
    const int j0 = lo + tile * KT;
    f32x16 sc[kSub];
#pragma unroll
    for (int t = 0; t < kSub; ++t)
#pragma unroll
      for (int u = 0; u < 16; ++u) sc[t][u] = 0.0f;
#pragma unroll
    for (int st = 0; st < kSteps; ++st)
#pragma unroll
      for (int t = 0; t < kSub; ++t) {
        const int row = t * 32 + col;
        const u32x4 kf = *(const u32x4 *)&sk[buf][row * D + ((2 * st + hi) ^ k_swizzle<D>(col)) * 8];
        sc[t] = T::mfma32(kf, qf[st], sc[t]);
      }
    if (masked) {
#pragma unroll
      for (int t = 0; t < kSub; ++t) {
        const int up = pos - j0 - 32 * t;
        uint32_t own = first_bits(up + 1) & (uint32_t)(there >> (32 * t));   // the row's slots, as bits
        if (a.window > 0) own &= ~first_bits(up + 1 - a.window);
        own >>= hi * 4;
#pragma unroll
        for (int u = 0; u < 16; ++u)
          if (!(own & (1u << slot32(u, 0)))) sc[t][u] = -INFINITY;
      }
    }
    float top = sc[0][0];
#pragma unroll
    for (int t = 0; t < kSub; ++t)
#pragma unroll
      for (int u = t == 0 ? 1 : 0; u < 16; ++u) top = fmaxf(top, sc[t][u]);
    top *= c;
    if (__any(top > m_run + (kManyLazy + T::kShift))) {
      const float m_new = fmaxf(m_run, half_max(top) - T::kShift);
      const float alpha = m_new == -INFINITY ? 1.0f : fast_exp2(m_run - m_new);
      l_run *= alpha;
      m_run = m_new;
#pragma unroll
      for (int t = 0; t < kCols; ++t) acc[t] *= alpha;
    }
    const float m_use = m_run == -INFINITY ? 0.0f : m_run;
    u32x4 pf[kSub][2];
    float sum = 0.0f;
#pragma unroll
    for (int t = 0; t < kSub; ++t)
#pragma unroll
      for (int u = 0; u < 16; u += 2) {
        const float x = fast_exp2(__builtin_fmaf(sc[t][u], c, -m_use)), y = fast_exp2(__builtin_fmaf(sc[t][u + 1], c, -m_use));
        sum += x + y;
        pf[t][u >> 3][(u & 7) >> 1] = T::pack(x, y);
      }
    l_run += sum;

    // V^T operand of slots 16 ks .. of sub-tile t, columns 32 n ..: two transposing reads
#pragma unroll
    for (int t = 0; t < kSub; ++t)
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int n = 0; n < kCols; ++n) {
          const int l16 = lane & 15, rr = hi * 4 + (l16 >> 2), row = t * 32 + ks * 16 + rr;
          const int p = n * 4 + ((lane >> 4) & 1) * 2 + ((l16 & 3) >> 1), in = (l16 & 1) * 4;
          const uint16_t *x = &sv[buf][row * D + (p ^ v_swizzle<D>(rr)) * 8 + in];
          const s16x4 u = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)x);
          const s16x4 w = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)(x + 8 * D));
          const u32x2 ub = __builtin_bit_cast(u32x2, u), wb = __builtin_bit_cast(u32x2, w);
          acc[n] = T::mfma32((u32x4){ub.x, ub.y, wb.x, wb.y}, pf[t][ks], acc[n]);
        }
  };
  uint64_t there_next = 0;
  const auto turn = [&](int buf, int tile) {
    if (tile + kBufs - 1 < tiles) fetch(tile + kBufs - 1);
    const int j0 = lo + tile * KT;
    const uint64_t there = there_next;
    there_next = there_at(tile + 1);
    const bool masked = there != ~(uint64_t)0 || j0 + KT - 1 > first_pos ||
                        (a.window > 0 && j0 <= last_pos - a.window);
    if (masked) {
      clear(buf, tile, there);
      __syncthreads();
    }
    if (!idle) step(masked, buf, tile, there);
    if (tile % kChunk == 0 && tile + kChunk < tiles) {      // a chunk ahead of the first fetch from it
      page_put(tile / kChunk + 1);
      page_load(tile / kChunk + 2);
    }
    if (tile + 1 < tiles) arrive(tile + 1);
    __syncthreads();
  };
  if (tiles > 0) {
    if (tid == 0) sh_odd = 0;
    page_load(0);
    page_put(0);
    page_load(1);
    __syncthreads();
    for (int t = 0; t < kBufs - 1 && t < tiles; ++t) fetch(t);
    arrive(0);
    __syncthreads();
  }
  if (tiles > 0) there_next = there_at(0);
  for (int tile = 0; tile < tiles; ++tile) turn(tile % kBufs, tile);
  if (tiles > 0 && sh_odd) {
    // p is above 0 wherever a row sees a slot: an infinity or NaN in it is the sum
    const int stop = lo + tiles * KT < end ? lo + tiles * KT : end;
    for (int j = lo; j < stop; ++j) {
      if (!(j > first_pos || (a.window > 0 && j <= last_pos - a.window))) continue;
      const SlotPlace pl = slot_place(a.c, trow, (uint32_t)j);
      const int64_t o = place_offset(a.c, pl);
      if (o < 0 || j > pos || (a.window > 0 && j <= pos - a.window)) continue;
#pragma unroll
      for (int n = 0; n < kCols; ++n)
#pragma unroll
        for (int k = 0; k < 16; k += 4) {
          const int d = n * 32 + slot32(k, hi);
          const char *e = vbase + o + d * BITS / 8;
          u32x2 x;
          if (E2M1) {
            const uint32_t w = *(const uint16_t *)e, power = a.c.v_power[(uint64_t)place_number(a.c, pl, h) * kBlocks + n];
            x = (u32x2){T::template from_e2m1<0>(w, power), T::template from_e2m1<1>(w, power)};
          } else if (E4M3) {
            const uint32_t w = *(const uint32_t *)e;
            x = (u32x2){T::template from_e4m3<false>(w), T::template from_e4m3<true>(w)};
          } else {
            x = *(const u32x2 *)e;
          }
          acc[n][k] += nonfinite_lo<T>(x.x);
          acc[n][k + 1] += nonfinite_hi<T>(x.x);
          acc[n][k + 2] += nonfinite_lo<T>(x.y);
          acc[n][k + 3] += nonfinite_hi<T>(x.y);
        }
    }
  }

  l_run = half_sum(l_run);
  if (!real) return;
  const int64_t at = (sp.t0 + tok) * heads + h * G + g;
  const float vs = E4M3 ? a.c.v_scale[h] : 1.0f;
  const bool any = l_run > 0.0f || l_run != l_run;
  if (a.nsplit > 1) {
    const int64_t part = (int64_t)split * a.tokens * heads + at;
    if (hi == 0) a.part_ml[part] = make_float2(m_run, l_run);
    if (!any) return;
    float *po = a.part_o + part * D;
#pragma unroll
    for (int n = 0; n < kCols; ++n)
#pragma unroll
      for (int k = 0; k < 16; k += 4)
        *(f32x4 *)(po + n * 32 + slot32(k, hi)) =
            (f32x4){acc[n][k] * vs, acc[n][k + 1] * vs, acc[n][k + 2] * vs, acc[n][k + 3] * vs};
  } else {
    if (hi == 0) a.lse[at] = any ? (m_run + __log2f(l_run)) * kLn2 : -INFINITY;
    const float mul = any ? vs / l_run : 0.0f;
    char *out = a.out + at * D * 2;
#pragma unroll
    for (int n = 0; n < kCols; ++n)
#pragma unroll
      for (int k = 0; k < 16; k += 4)
        *(u32x2 *)(out + (n * 32 + slot32(k, hi)) * 2) =
            (u32x2){T::pack(acc[n][k] * mul, acc[n][k + 1] * mul), T::pack(acc[n][k + 2] * mul, acc[n][k + 3] * mul)};
  }
}

// Column sums.  Grid: slot tiles x heads x sequences x row splits.  A wave holds K of 64 slots and
// reads each Q tile from LDS once for both halves: with 32 the LDS reads alone would take as long
// as the products.
template <class T, int BITS, int D>
__global__ __launch_bounds__(kManyThreads, D > 128 ? 1 : 2) void attend_sums_kernel(AttendArgs a) {
  constexpr bool E4M3 = BITS == 8, E2M1 = BITS == 4;
  constexpr int QT = 64;                             // rows of a tile
  constexpr int kSteps = D / 16, kPieces = D / 8;
  constexpr int kLoads = QT * kPieces / kManyThreads;
  __shared__ __align__(16) uint16_t sq[2][QT * D];
  __shared__ __align__(16) float sl[2][QT];          // -lse of the rows in log2 units
  __shared__ __align__(16) int sp_[2][QT];           // their slots

  const int H = a.c.heads, G = a.group;
  const int64_t heads = (int64_t)H * G;
  const int nst = (a.max_len + kSumSlotsTile - 1) / kSumSlotsTile;
  int b = blockIdx.x;
  const int h = b % H;
  b /= H;
  const int st = b % nst;
  b /= nst;
  const int s = b % a.c.seqs, rsplit = b / a.c.seqs;
  const int tid = threadIdx.x, lane = tid & 63, col = lane & 31, hi = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const SeqSpan sp = seq_span(a.starts, a.c.lens, s, a.tokens, a.max_q, a.max_len);
  const int slot0 = st * kSumSlotsTile;
  if (slot0 >= sp.n) return;
  const int wave0 = slot0 + wave * 64;               // the wave's slots
  int j[2];
  SlotPlace pl[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    j[x] = wave0 + x * 32 + col;
    pl[x] = SlotPlace{-1, 0};
    if (j[x] < sp.n) pl[x] = slot_place(a.c, a.c.table + (int64_t)s * a.c.table_stride, (uint32_t)j[x]);
  }
  // tokens that see any slot of the tile
  int i0 = slot0 - sp.first, i1 = sp.m;
  i0 = i0 < 0 ? 0 : i0;
  if (a.window > 0) {
    const int64_t e = (int64_t)slot0 + kSumSlotsTile - 1 + a.window - sp.first;
    i1 = e < i1 ? (int)e : i1;
  }
  const int r0 = i0 * G, r1 = i1 > i0 ? i1 * G : i0 * G;
  int tiles = (r1 - r0 + QT - 1) / QT;
  const int per = (tiles + a.nrow - 1) / a.nrow;
  const int tile0 = rsplit * per < tiles ? rsplit * per : tiles;
  const int tile1 = tile0 + per < tiles ? tile0 + per : tiles;
  u32x4 kf[2][kSteps];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    if (tile0 >= tile1) break;       // no row sees the tile
    const int64_t o = place_offset(a.c, pl[x]);
    const char *kp = a.c.k + (int64_t)h * a.c.head_stride + (o < 0 ? 0 : o);
    const uint8_t *powers = E2M1 ? a.c.k_power + (uint64_t)place_number(a.c, pl[x], h) * (D / kPowerBlock) : nullptr;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      if (E2M1) kf[x][i] = widen_e2m1<T>(*(const uint32_t *)(kp + i * 8 + hi * 4), powers[i / 2]);
      else if (E4M3) kf[x][i] = widen_e4m3<T>(*(const u32x2 *)(kp + i * 16 + hi * 8));
      else kf[x][i] = *(const u32x4 *)(kp + i * 32 + hi * 16);
    }
  }
  const float c = E4M3 ? a.scale_log2 * a.c.k_scale[h] : a.scale_log2;

  u32x4 gq[kLoads];
  float gl = 0.0f;
  int gp = 0;
  const auto fetch = [&](int tile) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int id = tid + i * kManyThreads, row = id / kPieces, p = id - row * kPieces, r = r0 + tile * QT + row;
      const int tok = (int)fast_div(a.gdiv, (uint32_t)r), g = r - tok * G;
      gq[i] = (u32x4){0, 0, 0, 0};
      if (r < r1) gq[i] = *(const u32x4 *)(a.q + (sp.t0 + tok) * a.q_stride + ((int64_t)(h * G + g) * D) * 2 + p * 16);
    }
    if (tid < QT) {
      const int r = r0 + tile * QT + tid;
      const int tok = (int)fast_div(a.gdiv, (uint32_t)r), g = r - tok * G;
      float l = -INFINITY;       // a row that is not there, or sees nothing, gives 0
      if (r < r1) {
        l = -kLog2e * a.lse[(sp.t0 + tok) * heads + h * G + g];
        if (l == INFINITY) l = -INFINITY;
      }
      gl = l;
      gp = r < r1 ? sp.first + tok : -1;
    }
  };
  const auto store = [&](int buf) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int id = tid + i * kManyThreads, row = id / kPieces, p = id - row * kPieces;
      *(u32x4 *)&sq[buf][row * D + (p ^ k_swizzle<D>(row)) * 8] = gq[i];
    }
    if (tid < QT) {
      sl[buf][tid] = gl;
      sp_[buf][tid] = gp;
    }
  };
  const uint32_t reach = a.window > 0 ? (uint32_t)a.window : 0x80000000u;
  // One tile.  Without a branch in it the products of the second 32 rows go under the first's exponentials.
  const auto add_tile = [&](auto masked, int buf, float (&part)[2]) {
#pragma unroll
    for (int t = 0; t < QT / 32; ++t) {
      f32x16 sc[2];
#pragma unroll
      for (int u = 0; u < 16; ++u) sc[0][u] = sc[1][u] = 0.0f;
      const int row = t * 32 + col;
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const u32x4 qf = *(const u32x4 *)&sq[buf][row * D + ((2 * i + hi) ^ k_swizzle<D>(col)) * 8];
        sc[0] = T::mfma32(qf, kf[0][i], sc[0]);
        sc[1] = T::mfma32(qf, kf[1][i], sc[1]);
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f32x4 l = *(const f32x4 *)&sl[buf][t * 32 + q * 8 + hi * 4];
        float p[2][4];
        u32x4 at = (u32x4){0, 0, 0, 0};
        if (decltype(masked)::value) at = *(const u32x4 *)&sp_[buf][t * 32 + q * 8 + hi * 4];
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            float z = __builtin_fmaf(sc[x][q * 4 + u], c, l[u]);
            // the row's slot less this one: 0 .. window - 1, and below 0 a large number
            if (decltype(masked)::value) z = at[u] - (uint32_t)j[x] < reach ? z : -INFINITY;
            p[x][u] = fast_exp2(z);
          }
#pragma unroll
        for (int x = 0; x < 2; ++x) part[x] += (p[x][0] + p[x][1]) + (p[x][2] + p[x][3]);
      }
    }
  };
  // a tile's terms are added up first: the running sums take one rounding for each
  float sum[2] = {0.0f, 0.0f}, low[2] = {0.0f, 0.0f};   // and what those roundings lost
  if (tile0 < tile1) {
    fetch(tile0);
    store(0);
    __syncthreads();
  }
  for (int tile = tile0; tile < tile1; ++tile) {
    const int buf = (tile - tile0) & 1;
    const bool more = tile + 1 < tile1;
    if (more) fetch(tile + 1);
    // slots of the first and last row of the tile
    const int ra = r0 + tile * QT, rb = ra + QT < r1 ? ra + QT - 1 : r1 - 1;
    const int pa = sp.first + (int)fast_div(a.gdiv, (uint32_t)ra), pb = sp.first + (int)fast_div(a.gdiv, (uint32_t)rb);
    // of the wave's own 64 slots: none that a row of the tile sees, or some that some row does not see (a row
    // that is not there sees none: its zeros times an infinite key are not)
    const bool none = wave0 > pb || (a.window > 0 && wave0 + 63 <= pa - a.window);
    const bool masked = wave0 + 63 > pa || (a.window > 0 && wave0 <= pb - a.window) || ra + QT > r1;
    float part[2] = {0.0f, 0.0f};
    if (!none) {
      if (masked) add_tile(std::true_type{}, buf, part);
      else add_tile(std::false_type{}, buf, part);
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const float y = part[x] - low[x], z = sum[x] + y;
      low[x] = (z - sum[x]) - y;
      sum[x] = z;
    }
    if (more) store(buf ^ 1);
    __syncthreads();
  }
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const float w = half_sum(sum[x]);
    if (j[x] >= sp.n || hi) continue;
    if (a.nrow > 1) {
      a.part_w[((int64_t)rsplit * a.c.seqs * H + (int64_t)s * H + h) * a.max_len + j[x]] = w;
    } else if (pl[x].page >= 0) {
      float *to = a.c.weights + ((int64_t)pl[x].page * H + h) * a.c.page.d + pl[x].row;
      *to = a.decay != 0.0f ? a.decay * *to + w : w;
    }
  }
}

template <class T, int BITS>
void launch_many(const AttendArgs &a, int dim, dim3 grid, hipStream_t st) {
  if (dim == 64) attend_many_kernel<T, BITS, 64><<<grid, kManyThreads, 0, st>>>(a);
  else if (dim == 96) attend_many_kernel<T, BITS, 96><<<grid, kManyThreads, 0, st>>>(a);
  else if (dim == 128) attend_many_kernel<T, BITS, 128><<<grid, kManyThreads, 0, st>>>(a);
  else attend_many_kernel<T, BITS, 256><<<grid, kManyThreads, 0, st>>>(a);
}
template <class T, int BITS>
void launch_sums(const AttendArgs &a, int dim, dim3 grid, hipStream_t st) {
  if (dim == 64) attend_sums_kernel<T, BITS, 64><<<grid, kManyThreads, 0, st>>>(a);
  else if (dim == 96) attend_sums_kernel<T, BITS, 96><<<grid, kManyThreads, 0, st>>>(a);
  else if (dim == 128) attend_sums_kernel<T, BITS, 128><<<grid, kManyThreads, 0, st>>>(a);
  else attend_sums_kernel<T, BITS, 256><<<grid, kManyThreads, 0, st>>>(a);
}

}  // namespace kmi
