// paged_few.h -- attention of few rows over a paged cache (one to a few new tokens a sequence).
//
//   out[t, g] = sum_j p_j v_j,   p_j = exp(z_j - lse),  z_j = scale <q[t, g], k_j>,
//   over the slots j that token t sees: j <= its own slot, and j > its slot - window.
//
// The rows of a key/value head are its `group` query heads times the sequence's new tokens; up to
// 32 of them share one pass over the head's slots, so the cache is read once and HBM bounds it.
// The slots of all sequences and heads are dealt to as many work-groups as the device holds, in equal
// runs of tiles of 32 slots; a work-group's four waves take every fourth tile of its run.
//
//  * No LDS between HBM and the matrix instructions.  With S^T = K Q^T the A operand is rows of K
//    as they lie in memory, and the result leaves lane l with row l % 16 and slots 4 (l / 16) + r
//    of each 16.  Counting a tile's 32 slots in that order makes the packed p the B operand of
//    O^T = V^T P^T as it stands.  V^T wants eight slots of one column in a lane: each lane loads
//    the same few columns of its eight slots and swaps halves of registers (v_perm).
//  * K of the next tile is loaded once S is formed and V of the next once O is updated, into the
//    registers just read: each wave keeps about a tile's bytes in flight at all times.
//  * The running maximum moves only when a score passes it by 2^8 (one branch per tile), so the
//    sums and p stay below 2^8 times what they would be; sums are in 32 bits, of p as it is.  p is
//    rounded to the cache's 16-bit type (8-bit caches: q's) for the product with V: the matrix
//    instructions take two 16-bit operands, or two fp32 ones at a sixteenth of the rate.  The output's
//    error against 64 bits goes from its own rounding's 0.0017 to 0.0022 by it (bf16); 4-bit caches of up to 16
//    rows have the remainder of p multiplied as well.
//  * HBM bounds it: 64 sequences of 5,120 slots (bf16, 16 rows a head) read 1.34 GB in 242 us, 5.6 TB/s
//    with both passes; 131,071 slots of one sequence 5.4 TB/s and 5 us of the second pass.
//  * 4-bit caches: a head's row is half a line or less, and a lane's piece of it is 4 or 8 bytes, so that loads as above
//    would be bound by their number.  A tile's rows are loaded 16 bytes a lane and pass through LDS, a wave's own, to
//    the lanes that use them (codes become 16-bit values under their block's power in one instruction a pair); two
//    tiles of a wave are on their way at a time.  Where the device is filled all the same, neighbouring heads whose
//    rows make up a 128-byte line go to the same work-group, whose waves load whole lines for each other; all heads of
//    the same slots run on one XCD, whose L2 then holds the lines of the powers that they share.  64 sequences of up
//    to 8,192 slots with 4 drafts (8 heads of 128): 129 us without, 85 so, 90 with p in two parts; 131,071 slots of one sequence 56 and 44.
//  * Slots that no row may see (past the length, of a page that the table lacks) get a zero V.
//    Slots that some rows see and others do not are only in the tiles of the new tokens and at
//    the window's edge; if such a tile holds an infinity or NaN in V, it is added after the
//    products, to the rows that see it (0 times infinity would reach the others).  So is every infinity or NaN of a
//    4-bit cache of up to 16 rows, whose tiles are multiplied with p's remainder too: one in each page of 131,071 slots
//    takes 99 us in place of 43.
#pragma once

#include <atomic>

#include "paged.h"

namespace kmi {

constexpr int kFewWaves = 4;
constexpr int kFewThreads = kFewWaves * kWave;
constexpr int kFewTile = 32;       // slots of a wave's tile
constexpr int kFewBlock = 1024;    // slots whose addresses are held in LDS at a time
constexpr int kScoreHeld = 8192;   // scores held in LDS for 16 rows
constexpr float kLazy = 8.0f;      // log2 of what a score may pass the running maximum by

// V columns of a lane: pieces of W consecutive columns, column base + (l % 16) W + t.
template <int D> struct VPieces;
template <> struct VPieces<64> { static constexpr int n = 1; static constexpr int w[2] = {4, 0}; };
template <> struct VPieces<96> { static constexpr int n = 2; static constexpr int w[2] = {4, 2}; };
template <> struct VPieces<128> { static constexpr int n = 1; static constexpr int w[2] = {8, 0}; };
template <> struct VPieces<256> { static constexpr int n = 2; static constexpr int w[2] = {8, 8}; };

__device__ __forceinline__ float xor_max(float v) {   // over the four lanes of a row
  v = fmaxf(v, __shfl_xor(v, 16));
  return fmaxf(v, __shfl_xor(v, 32));
}
__device__ __forceinline__ float xor_sum(float v) {
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}

template <class T, int BITS, int D, int NR>
struct FewRows {
  static constexpr bool E4M3 = BITS == 8, E2M1 = BITS == 4;
  static constexpr int kBytes = E4M3 ? 1 : 2;           // of an element (e2m1: two to a byte)
  static constexpr int kSteps = D / 32;                 // matrix steps along the head dimension
  static constexpr int kTiles = D / 16;                 // 16-column tiles of O^T
  static constexpr int kKRegs = (E2M1 ? 1 : E4M3 ? 2 : 4) * kSteps;
  static constexpr int kVRegs = E2M1 ? VPieces<D>::n : D / 16 * kBytes / 4 > 0 ? (D / 16 * kBytes + 3) / 4 : 1;   // registers of a slot's columns
  static constexpr int kPad = D + 4;                    // floats of a row in LDS: rows four banks apart

  uint32_t kr[2][kKRegs];
  uint32_t vr[8][kVRegs];
  // e2m1: the powers of the lane's blocks, of K the one of its first columns and, if there are two, of its last
  static constexpr int kKPowers = D == 96 || D == 256 ? 2 : 1;
  uint32_t kp[2][kKPowers], vp[8][VPieces<D>::n];

  // e2m1: a tile's keys, values and powers pass through LDS of the wave's own.  Neighbouring lanes load neighbouring
  // blocks of a slot (not a slot a lane, the operands' own order: four times the addresses to look up), the keys are
  // read back as the A operand and the values as eight slots of a lane's columns.
  static constexpr int kBlocks = D / kPowerBlock, kLoads = E2M1 ? (32 * kBlocks + kWave - 1) / kWave : 1;
  static constexpr int kGroup = 36;                     // words of an 8-column group of V, a slot each and a pad: no two lanes' banks meet
  static constexpr int kStageV = 16 * D, kStageP = kStageV + D / 8 * kGroup * 4;
  static constexpr int kStageBytes = E2M1 ? kStageP + 64 * kBlocks : 0;
  u32x4 ks[kLoads], vs[kLoads];
  u32x2 pw;
  // where block b of a slot's key lies, in 16 bytes: the 16 slots that are read together meet all banks
  static __device__ __forceinline__ int key_unit(int slot, int b) {
    const int x = D == 64 ? (slot >> 3) & 1 : D == 128 ? (slot >> 2) & 3 : D == 256 ? (slot >> 1) & 7 : 0;
    return slot * kBlocks + (b ^ x);
  }

  // 8-bit rows of a multiple of 64 bytes: a lane's 16 bytes are the operands of two matrix steps,
  // columns 64 s + 16 (l / 16) + 8 u .. of steps 2 s + u.  Any order of the columns will do that Q shares.
  static constexpr bool kWide = E4M3 && D % 64 == 0;
  // 4-bit ones: a lane's columns lie in a row (D = 256: in two), D / 8 bytes.
  static __device__ __forceinline__ int step_column(int s, int q) {
    if (E2M1) return D == 256 ? (s >> 2) * 128 + q * 32 + (s & 3) * 8 : q * (D / 4) + s * 8;
    return kWide ? (s >> 1) * 64 + q * 16 + (s & 1) * 8 : s * 32 + q * 8;
  }

  // K rows of the tile: lane l has slot l % 16 of each 16, columns step_column(s, l / 16) ..+8 of step s.
  template <bool FAR>
  __device__ __forceinline__ void load_k(const char *base, const int64_t *off, int at) {
    const int lane = threadIdx.x & (kWave - 1), row = lane & 15, q = lane >> 4;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      int64_t o = off[at + 16 * t + row];
      o = o < 0 ? 0 : o;
      const char *p = base + o + step_column(0, q) * kBytes;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        if (kWide) {
          if (s & 1) continue;
          const u32x4 w = load_once<u32x4, FAR>((p + s * 32));
#pragma unroll
          for (int u = 0; u < 4; ++u) kr[t][(2 * s + u) % kKRegs] = w[u];
        } else if (E4M3) {
          const u32x2 w = load_once<u32x2, FAR>((p + s * 32));
          kr[t][2 * s] = w.x;
          kr[t][2 * s + 1] = w.y;
        } else {
          const u32x4 w = load_once<u32x4, FAR>((p + s * 64));
#pragma unroll
          for (int u = 0; u < 4; ++u) kr[t][4 * s + u] = w[u];
        }
      }
    }
  }

  // V: lane l has slots 4 (l / 16) + i of the first 16 (i < 4) and of the second (i >= 4).
  template <bool FAR>
  __device__ __forceinline__ void load_v(const char *base, const int64_t *off, int at) {
    const int lane = threadIdx.x & (kWave - 1), c = lane & 15, q = lane >> 4;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      int64_t o = off[at + (i >> 2) * 16 + q * 4 + (i & 3)];
      o = o < 0 ? 0 : o;
      const char *p = base + o;
      int reg = 0, col = 0;
#pragma unroll
      for (int n = 0; n < VPieces<D>::n; ++n) {
        const int w = VPieces<D>::w[n], b = w * kBytes;
        const char *e = p + (col + c * w) * kBytes;
        if (b == 16) {
          const u32x4 x = load_once<u32x4, FAR>(e);
#pragma unroll
          for (int u = 0; u < 4; ++u) vr[i][(reg + u) % kVRegs] = x[u];
          reg += 4;
        } else if (b == 8) {
          const u32x2 x = load_once<u32x2, FAR>(e);
          vr[i][reg % kVRegs] = x.x;
          vr[i][(reg + 1) % kVRegs] = x.y;
          reg += 2;
        } else if (b == 4) {
          vr[i][reg % kVRegs] = load_once<uint32_t, FAR>(e);
          reg += 1;
        } else {
          vr[i][reg % kVRegs] = load_once<uint16_t, FAR>(e);
          reg += 1;
        }
        col += 16 * w;
      }
    }
  }

  // A wave's share of the blocks of a tile: 2^lg waves, each with a head of its own, load the slots' blocks of all their
  // heads, which lie side by side, so that a request to L2 is for a whole line (L1 has so many of them under way).
  // place: this wave's among them.
  struct Share {
    int lg, place;
    __device__ __forceinline__ void item(int n, int *slot, int *head, int *b) const {
      const int i = n * kWave + (int)(threadIdx.x & (kWave - 1)), at = i / kBlocks;
      *b = i - at * kBlocks;
      *head = at & ((1 << lg) - 1);
      *slot = (at >> lg) + place * (32 >> lg);
    }
    static __device__ __forceinline__ bool has(int n) {        // D = 96: the last half round is empty
      return 32 * kBlocks % kWave == 0 || n * kWave + (int)(threadIdx.x & (kWave - 1)) < 32 * kBlocks;
    }
  };
  // A tile's K, V and powers on their way.  kbase, vbase: of the first head; number: the slots' numbers among its powers.
  template <bool FAR>
  __device__ __forceinline__ void load_staged(const Share &sh, int64_t head_stride, const char *kbase, const char *vbase, const int64_t *off,
                                              const uint8_t *kpow, const uint8_t *vpow, const uint32_t *number, int at) {
    const int lane = threadIdx.x & (kWave - 1);
#pragma unroll
    for (int n = 0; n < kLoads; ++n) {
      int slot, head, b;
      sh.item(n, &slot, &head, &b);
      if (!sh.has(n)) continue;
      int64_t o = off[at + slot];
      o = (o < 0 ? 0 : o) + head * head_stride + b * 16;
      ks[n] = load_once<u32x4, FAR>(kbase + o);
      vs[n] = load_once<u32x4, FAR>(vbase + o);
    }
    // a slot's powers, of K by the lower lanes and of V by the upper ones
    const uint8_t *e = (lane < 32 ? kpow : vpow) + (uint64_t)number[at + (lane & 31)] * kBlocks;
    if (D == 64) pw.x = load_once<uint16_t, FAR>(e);
    else if (D == 96) pw.x = load_once<uint8_t, FAR>(e) | (uint32_t)load_once<uint8_t, FAR>(e + 1) << 8 | (uint32_t)load_once<uint8_t, FAR>(e + 2) << 16;
    else if (D == 128) pw.x = load_once<uint32_t, FAR>(e);
    else pw = load_once<u32x2, FAR>(e);
  }
  // What has arrived to LDS: blocks to the places of their heads, from `all` on, and powers to the wave's own.
  __device__ __forceinline__ void put_staged(const Share &sh, char *all, char *stage) {
    const int lane = threadIdx.x & (kWave - 1);
    uint8_t *const sp = (uint8_t *)(stage + kStageP);   // K [slot][block], then V [block][slot]
#pragma unroll
    for (int n = 0; n < kLoads; ++n) {
      int slot, head, b;
      sh.item(n, &slot, &head, &b);
      if (!sh.has(n)) continue;
      char *const to = all + head * kStageBytes;
      ((u32x4 *)to)[key_unit(slot, b)] = ks[n];
      uint32_t *const sv = (uint32_t *)(to + kStageV);
#pragma unroll
      for (int u = 0; u < 4; ++u) sv[(4 * b + u) * kGroup + slot] = vs[n][u];
    }
    const int slot = lane & 31;
    const int v = lane >> 5;                            // K: bytes 0 .. of the slot; V: a block's bytes 32 apart
#pragma unroll
    for (int b = 0; b < kBlocks; ++b)
      sp[v ? 32 * (kBlocks + b) + slot : slot * kBlocks + b] = (uint8_t)((b < 4 ? pw.x : pw.y) >> (8 * (b & 3)));
  }
  // K and its powers from there.
  __device__ __forceinline__ void take_keys(const char *stage) {
    const int lane = threadIdx.x & (kWave - 1), row = lane & 15, q = lane >> 4;
    const uint8_t *const sp = (const uint8_t *)(stage + kStageP);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int slot = 16 * t + row;
      if (D == 64) {
        const u32x2 w = *(const u32x2 *)(stage + key_unit(slot, q >> 1) * 16 + (q & 1) * 8);
        kr[t][0] = w.x;
        kr[t][1 % kKRegs] = w.y;
      } else if (D == 96) {
#pragma unroll
        for (int u = 0; u < 3; ++u) kr[t][u % kKRegs] = *(const uint32_t *)(stage + slot * 48 + q * 12 + u * 4);
      } else {
#pragma unroll
        for (int s = 0; s < kSteps; s += 4) {
          const u32x4 w = ((const u32x4 *)stage)[key_unit(slot, q + s)];
#pragma unroll
          for (int u = 0; u < 4; ++u) kr[t][(s + u) % kKRegs] = w[u];
        }
      }
      kp[t][0] = sp[slot * kBlocks + step_column(0, q) / kPowerBlock];
      if (kKPowers > 1) kp[t][kKPowers - 1] = sp[slot * kBlocks + step_column(kSteps - 1, q) / kPowerBlock];
    }
  }
  // V as load_v has it: slots 4 q + i of the first 16 and of the second.
  __device__ __forceinline__ void take_staged(const char *stage) {
    const int lane = threadIdx.x & (kWave - 1), c = lane & 15, q = lane >> 4;
    const uint32_t *const sv = (const uint32_t *)(stage + kStageV);
    const uint8_t *const sp = (const uint8_t *)(stage + kStageP) + 32 * kBlocks;
    int base = 0;
#pragma unroll
    for (int n = 0; n < VPieces<D>::n; ++n) {
      const int w = VPieces<D>::w[n], col = base + c * w;       // the piece's first
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const u32x4 x = *(const u32x4 *)(sv + col / 8 * kGroup + 16 * t + 4 * q);
        const uint32_t p = *(const uint32_t *)(sp + col / kPowerBlock * 32 + 16 * t + 4 * q);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          vr[4 * t + i][n % kVRegs] = w == 8 ? x[i] : x[i] >> (col & 7) * 4;
          vp[4 * t + i][n] = (p >> (8 * i)) & 0xffu;
        }
      }
      base += 16 * w;
    }
    __builtin_amdgcn_wave_barrier();
  }

  __device__ __forceinline__ u32x4 k_frag(int t, int s) const {
    if (E2M1) {
      uint32_t power = kp[t][0];
      if (D == 256) power = kp[t][(s >> 2) % kKPowers];
      if (D == 96) {
        const int q = (threadIdx.x & (kWave - 1)) >> 4;
        power = (3 * q + s) >> 2 == (3 * q) >> 2 ? kp[t][0] : kp[t][kKPowers - 1];
      }
      return widen_e2m1<T>(kr[t][s], power);
    }
    if (E4M3) return widen_e4m3<T>((u32x2){kr[t][2 * s], kr[t][2 * s + 1]});
    return (u32x4){kr[t][4 * s], kr[t][4 * s + 1], kr[t][4 * s + 2], kr[t][4 * s + 3]};
  }

  // Columns 2 m and 2 m + 1 of slot i's W columns of piece n, as a 16-bit pair.
  __device__ __forceinline__ uint32_t v_pair(int i, int n, int m) const {
    if (E2M1) return e2m1_pair<T>(vr[i][n % kVRegs], vp[i][n], m);
    if (!E4M3) return vr[i][(n ? VPieces<D>::w[0] / 2 : 0) + m];
    const int at = (n ? VPieces<D>::w[0] : 0) + 2 * m;    // first of the two bytes
    const uint32_t w = vr[i][at / 4];
    return (at & 2) ? T::template from_e4m3<true>(w) : T::template from_e4m3<false>(w);
  }

  // A operands of column tiles 2 m and 2 m + 1 of piece n: one column of the lane's eight slots.
  __device__ __forceinline__ void v_frags(int n, int m, u32x4 &lo, u32x4 &hi) const {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t x = v_pair(2 * u, n, m), y = v_pair(2 * u + 1, n, m);
      lo[u] = __builtin_amdgcn_perm(y, x, 0x05040100u);
      hi[u] = __builtin_amdgcn_perm(y, x, 0x07060302u);
    }
  }
};

// A sequence's share of the few-rows work: its tiles of 32 slots from the first that any row sees.
struct FewSpan {
  SeqSpan sp;
  int lo, hi, tiles;         // slots [lo, hi), lo a multiple of the tile; at least one tile if there are rows
};
__device__ __forceinline__ FewSpan few_span(const AttendArgs &a, int s) {
  FewSpan f;
  f.sp = seq_span(a.starts, a.c.lens, s, a.tokens, a.max_q, a.max_len);
  f.lo = 0;
  if (a.window > 0 && f.sp.first - a.window + 1 > 0) f.lo = (f.sp.first - a.window + 1) & ~(kFewTile - 1);
  f.hi = f.sp.n < f.sp.first + f.sp.m ? f.sp.n : f.sp.first + f.sp.m;
  f.tiles = f.hi > f.lo ? (f.hi - f.lo + kFewTile - 1) / kFewTile : 1;
  if (f.sp.m == 0) f.tiles = 0;
  return f;
}
// All tiles of all sequences and heads in a line, sequence by sequence, head by head, are dealt to
// the work-groups in equal runs.  Every wave finds out for itself, from the lengths.
struct FewShare {
  uint32_t share;            // tiles of a work-group
  int s;                     // the sequence that holds tile `at` of the line (seqs: past the end)
  uint32_t base;             // the first of its tiles
  FewSpan span;              // of that sequence
};
__device__ __forceinline__ uint32_t share_of(uint32_t total, int wgs) {
  const uint32_t share = (total + wgs - 1) / wgs;
  return (share + kFewWaves - 1) / kFewWaves * kFewWaves;      // a tile for every wave
}
__device__ __forceinline__ int lane_of(int v, int lane) { return __builtin_amdgcn_readlane(v, lane); }
// A lane's sequence of 64 from s0 on: its span, and the line's tiles up to it.
struct FewLine {
  FewSpan f;
  uint32_t own, upto;
};
__device__ __forceinline__ FewLine few_line(const AttendArgs &a, int s0, uint32_t before, int heads) {
  const int s = s0 + (int)(threadIdx.x & (kWave - 1));
  FewLine r{};
  if (s < a.c.seqs) r.f = few_span(a, s);
  r.own = s < a.c.seqs ? (uint32_t)(r.f.tiles * heads) : 0u;
  r.upto = before + wave_scan_u32(r.own);
  return r;
}
// `note`: write down for the second pass where each sequence's tiles begin, and after them the share.  heads: those
// whose tiles are in the line, all of them or one.
__device__ __forceinline__ FewShare few_share(const AttendArgs &a, int heads, int wgs, int wg, bool note) {
  const int S = a.c.seqs, lane = threadIdx.x & (kWave - 1);
  FewLine line = few_line(a, 0, 0, heads);
  if (note && lane < S) a.line[lane] = line.upto - line.own;
  uint32_t total = lane_of(line.upto, kWave - 1);
  for (int s0 = kWave; s0 < S; s0 += kWave) {
    const FewLine next = few_line(a, s0, total, heads);
    if (note && s0 + lane < S) a.line[s0 + lane] = next.upto - next.own;
    total = lane_of(next.upto, kWave - 1);
  }
  FewShare r{share_of(total, wgs), S, total, {}};
  if (note && lane == 0) a.line[S] = r.share;
  const uint32_t at = (uint32_t)wg * r.share;
  for (int s0 = 0;;) {
    const uint64_t who = __ballot(at >= line.upto - line.own && at < line.upto);
    if (who) {
      const int l = __ffsll((unsigned long long)who) - 1;
      r.s = s0 + l;
      r.base = lane_of(line.upto - line.own, l);
      const FewSpan &f = line.f;
      r.span = FewSpan{{lane_of((int)f.sp.t0, l), lane_of(f.sp.m, l), lane_of(f.sp.n, l), lane_of(f.sp.first, l)},
                       lane_of(f.lo, l), lane_of(f.hi, l), lane_of(f.tiles, l)};
      break;
    }
    if ((s0 += kWave) >= S) break;
    line = few_line(a, s0, lane_of(line.upto, kWave - 1), heads);
  }
  return r;
}
// The work-groups [w0, w1] that share a (sequence, head), counted among those of the head if each has its own.
__device__ __forceinline__ void part_range(const AttendArgs &a, uint32_t share, uint32_t begin, int h, int tiles, int *w0, int *w1) {
  const uint32_t from = begin + (a.by_head ? 0u : (uint32_t)(h * tiles)), to = from + tiles;
  *w0 = (int)(from / share);
  *w1 = (int)((to - 1) / share);
}

// NW waves: 4, or 8 where one work-group has a short sequence's head to itself and nothing else
// would hide its latency.
// FAR: the call's keys and values, by its bounds, are more than the last-level cache holds, and pass it by.
template <class T, int BITS, int D, int NR, bool SCORES, int NW, bool FAR>
__global__ __launch_bounds__(NW * kWave, NW > 4 ? 2 : (D * NR > 128 || (SCORES && NR == 2) ? 1 : (BITS == 8 && NR == 1 ? 3 : 2))) void attend_few_kernel(AttendArgs a) {
  using F = FewRows<T, BITS, D, NR>;
  constexpr bool E4M3 = BITS == 8, E2M1 = BITS == 4;
  constexpr int kRows = 16 * NR;
  // 4-bit caches of up to 16 rows: p's rounding to 16 bits is multiplied with V too, so that of a row that few slots
  // decide no more is lost than the output's rounding (0.0017 of 64 bits in bf16, else 0.0023; up to half as much again
  // as that in single rows).  The products are there to be had: one token 1 to 3 % of the time, 16 rows 9.  32 rows
  // would take 14; the other caches' results are as they were.
  constexpr bool kBoth = E2M1 && NR == 1;
  constexpr int kHalfRows = NW / 2 * kRows;     // half the waves' rows
  // e2m1: heads that go together have two tiles in LDS in turn, so that one barrier a tile will do
  constexpr int kSets = E2M1 && !SCORES && NW == 4 && D < 256 ? 2 : 1;
  __shared__ __align__(16) union {
    struct {
      int64_t off[kFewBlock + kFewTile];
      char staged[E2M1 ? kSets * NW * F::kStageBytes : 16];
    };
    float o[kHalfRows * F::kPad];
  } sh;
  __shared__ float sh_m[NW / 2][kRows], sh_l[NW / 2][kRows];
  __shared__ uint32_t present[kFewBlock / kFewTile];     // a tile's slots that are there, as bits
  __shared__ int sh_odd;
  __shared__ uint32_t number[E2M1 ? kFewBlock + kFewTile : 1];     // the slots' among all powers
  // Kept scores of a block of slots, written out together: a store among the loads of every tile
  // would be waited for with them (22 us of 150 for a step of 32 conversations).
  __shared__ __align__(16) float scores[SCORES ? kScoreHeld * NR : 4];
  const int block = SCORES && a.score_rows * kFewBlock > kScoreHeld * NR
                        ? kScoreHeld * NR / a.score_rows / (kFewTile * NW) * (kFewTile * NW) : kFewBlock;

  const int H = a.c.heads, G = a.group;
  const int64_t heads = (int64_t)H * G;
  const int tid = threadIdx.x, lane = tid & (kWave - 1), col = lane & 15, q4 = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);

  // this work-group's run of tiles: from tile t0 of (s, h) on
  int s, h, t0;
  uint32_t left;
  FewSpan span;
  // A 4-bit row is less than a line of L2, and L1 has only so many requests under way, of a line or of a part of one.  A
  // work-group has a run of tiles of `hg` neighbouring heads, whose waves load for each other (FewRows::Share), and
  // the work-groups of all heads at the same slots run on one XCD.  64 conversations with 4 rows each, heads of 64
  // bytes side by side in a slot, took 127 us with a head's run anywhere, 107 on one XCD, 101 once neighbouring
  // lanes loaded neighbouring blocks, and 87 with whole lines; 84 where the pool has the heads apart.
  const int hg = E2M1 ? a.head_group : 1, wph = NW / hg;       // waves of a head
  const int lane_wave = E2M1 ? wave % wph : wave;              // this one's place among them
  int unit = 0, first_head = 0;
  if (E2M1) {
    const int groups = H / hg, units = gridDim.x / groups, paired = units / 8 * 8 * groups;
    const int b = blockIdx.x, k = b < paired ? b >> 3 : b - paired;
    first_head = k % groups * hg;
    unit = b < paired ? k / groups * 8 + (b & 7) : units / 8 * 8 + k / groups;
    h = first_head + wave / wph;
  }
  const int mine = E2M1 ? unit * H + h : (int)blockIdx.x;      // where its parts go
  if (a.whole) {
    s = mine / H;
    if (!E2M1) h = mine - s * H;
    t0 = 0;
    left = 0xffffffffu;
    span = few_span(a, s);
  } else if (E2M1) {
    const FewShare my = few_share(a, 1, gridDim.x / (H / hg), unit, blockIdx.x == 0 && wave == 0);
    if (my.s >= a.c.seqs) return;
    s = my.s;
    left = my.share;
    span = my.span;
    t0 = (int)((uint32_t)unit * my.share - my.base);
  } else {
    const FewShare my = few_share(a, H, gridDim.x, blockIdx.x, blockIdx.x == 0 && wave == 0);
    if (my.s >= a.c.seqs) return;
    s = my.s;
    left = my.share;
    span = my.span;
    const int at = (int)((uint32_t)blockIdx.x * my.share - my.base);
    h = at / span.tiles;
    t0 = at - h * span.tiles;
  }
  for (;;) {
  const SeqSpan &sp = span.sp;
  const int R = sp.m * G;
  if (R == 0) {              // `whole` only: the line has no such sequence
    if (a.whole) return;
    if (++s >= a.c.seqs) return;
    span = few_span(a, s);
    if (!E2M1) h = 0;
    continue;
  }
  const int hi = span.hi;
  const int t1 = (uint32_t)(span.tiles - t0) > left ? t0 + (int)left : span.tiles;
  const int c0 = span.lo + t0 * kFewTile;
  const int c1 = span.lo + t1 * kFewTile < hi ? span.lo + t1 * kFewTile : hi;
  // where a part goes: a run's first piece (2 wg), or the start of a longer one (2 wg + 1)
  const bool part = t0 > 0 || t1 < span.tiles;
  const int64_t part_at = ((int64_t)mine * 2 + (t0 > 0 ? 0 : 1)) * kRows;

  // rows of this lane: r = 16 nr + col, its token's slot (a padding row sees nothing)
  int pos[NR];
  u32x4 qf[NR][F::kSteps];
#pragma unroll
  for (int nr = 0; nr < NR; ++nr) {
    const int r = 16 * nr + col;
    const int tok = (int)fast_div(a.gdiv, (uint32_t)r), g = r - tok * G;
    pos[nr] = r < R ? sp.first + tok : -1;
    const char *qp = a.q + (sp.t0 + tok) * a.q_stride + (int64_t)(h * G + g) * D * 2;
#pragma unroll
    for (int st = 0; st < F::kSteps; ++st)
      qf[nr][st] = r < R ? *(const u32x4 *)(qp + F::step_column(st, q4) * 2) : (u32x4){0, 0, 0, 0};
  }
  // hidden scores are -inf before they are scaled: a negative factor's sign goes to Q, a zero one's
  // scores are zeros
  const float c0f = E4M3 ? a.scale_log2 * a.c.k_scale[h] : a.scale_log2;
  const float c = c0f == 0.0f ? 1.0f : fabsf(c0f);
  const uint32_t flip = c0f < 0.0f ? 0x80008000u : 0u, keep = c0f == 0.0f ? 0u : 0xffffffffu;
#pragma unroll
  for (int nr = 0; nr < NR; ++nr)
#pragma unroll
    for (int st = 0; st < F::kSteps; ++st)
#pragma unroll
      for (int u = 0; u < 4; ++u) qf[nr][st][u] = (qf[nr][st][u] ^ flip) & keep;

  float m_run[NR], l_run[NR];      // 2^m_run is the unit of the sums
  f32x4 acc[NR][F::kTiles];
#pragma unroll
  for (int nr = 0; nr < NR; ++nr) {
    m_run[nr] = -INFINITY;
    l_run[nr] = 0.0f;
#pragma unroll
    for (int t = 0; t < F::kTiles; ++t) acc[nr][t] = (f32x4){0, 0, 0, 0};
  }
  const char *kbase = a.c.k + (int64_t)h * a.c.head_stride;
  const char *vbase = a.c.v + (int64_t)h * a.c.head_stride;
  // from the first head's numbers
  const uint64_t past = E2M1 ? (uint64_t)(h - first_head) * a.c.page.d * (D / kPowerBlock) : 0;
  const uint8_t *kpow = a.c.k_power + past, *vpow = a.c.v_power + past;
  const int32_t *trow = a.c.table + (int64_t)s * a.c.table_stride;
  const int last_pos = sp.first + sp.m - 1;

  F f, f1;                   // f1: e2m1, the tile after the next
  // places in LDS by tile, then by head
  char *const all = sh.staged + (E2M1 ? lane_wave * hg * F::kStageBytes : 0), *const stage = all + (E2M1 ? wave / wph * F::kStageBytes : 0);
  const typename F::Share sharing{hg == 4 ? 2 : hg == 2 ? 1 : 0, wave / wph};
  const char *kfirst = a.c.k + (int64_t)first_head * a.c.head_stride, *vfirst = a.c.v + (int64_t)first_head * a.c.head_stride;
  bool odd = false;
  if (tid == 0) sh_odd = 0;
  // slots [from, from + cnt) from LDS: whole groups of four, as they lie in memory
  const auto flush = [&](int from, int cnt) {
    f32x4 *to = (f32x4 *)(a.scores + ((int64_t)(s * H + h) * (a.score_stride / 4) + (from >> 2)) * a.score_rows * 4);
    for (int i = tid; i < (cnt + 3) / 4 * a.score_rows; i += (NW * kWave)) to[i] = ((const f32x4 *)scores)[i];
  };
  for (int blk = c0; blk < c1; blk += block) {
    const int cnt = c1 - blk < block ? c1 - blk : block;
    const int ntile = (cnt + kFewTile - 1) / kFewTile;
    __syncthreads();
    if (SCORES && blk > c0) flush(blk - block, block);
    for (int i = tid; i < kFewBlock; i += (NW * kWave)) {
      const SlotPlace pl = i < cnt ? slot_place(a.c, trow, (uint32_t)(blk + i)) : SlotPlace{-1, 0};
      const int64_t o = place_offset(a.c, pl);
      sh.off[i] = o;
      if (E2M1) number[i] = place_number(a.c, pl, first_head);
      const uint64_t there = __ballot(o >= 0);
      if (lane == 0) {
        present[i / kFewTile] = (uint32_t)there;
        present[i / kFewTile + 1] = (uint32_t)(there >> 32);
      }
    }
    if (tid < kFewTile) sh.off[kFewBlock + tid] = -1;
    if (E2M1 && tid < kFewTile) number[kFewBlock + tid] = 0;
    __syncthreads();
    // after the last tile one row, again and again: loads without a condition let K be waited for alone
    const auto begin_of = [&](int tile) { return tile < ntile ? tile * kFewTile : kFewBlock; };
    const auto load_next = [&](F &f, int at) {
      f.template load_staged<FAR>(sharing, a.c.head_stride, kfirst, vfirst, sh.off, kpow, vpow, number, at);
    };
    const auto put = [&](F &f, int set) {
      const int from = set % kSets * NW * F::kStageBytes;
      f.put_staged(sharing, all + from, stage + from);
      if (hg > 1) __syncthreads();
      else __builtin_amdgcn_wave_barrier();
      return stage + from;
    };
    int tile = lane_wave;
    if constexpr (E2M1) {
      const auto step = [&](F &f, int tile, int next, const char *stage) {
#include "paged_few_tile.h"
      };
      // two tiles on their way: a 4-bit one alone is too few bytes
      load_next(f, begin_of(tile));
      __builtin_amdgcn_sched_barrier(0);
      load_next(f1, begin_of(tile + wph));
      __builtin_amdgcn_sched_barrier(0);
      // Always both tiles of a turn: with a way around the second, each would wait for the other's loads too.  All
      // waves take the same turns; in the last one a wave may be past the last tile.
      const int turns = (ntile + wph - 1) / wph;
      int i = 0;
      for (; i + 2 < turns; i += 2, tile += 2 * wph) {
        step(f, tile, begin_of(tile + 2 * wph), put(f, 0));
        step(f1, tile + wph, begin_of(tile + 3 * wph), put(f1, 1));
      }
      const char *at0 = put(f, 0);
      if (tile < ntile) step(f, tile, kFewBlock, at0);
      if (i + 1 < turns) {
        const char *at1 = put(f1, 1);
        if (tile + wph < ntile) step(f1, tile + wph, kFewBlock, at1);
      }
    } else {
      f.template load_k<FAR>(kbase, sh.off, begin_of(tile));
      __builtin_amdgcn_sched_barrier(0);
      f.template load_v<FAR>(vbase, sh.off, begin_of(tile));
      __builtin_amdgcn_sched_barrier(0);
      for (; tile < ntile; tile += NW) {
        const int next = begin_of(tile + NW);
#include "paged_few_tile.h"
      }
    }
  }

  __syncthreads();
  if (SCORES && c1 > c0) flush(c0 + (c1 - c0 - 1) / block * block, (c1 - c0 - 1) % block + 1);
  if (odd) sh_odd = 1;
  // other lanes read it: the hand-over's barriers come in between, unless each wave has a head of its own
  if (E2M1 && wph == 1) __syncthreads();
  // the waves' sums: the upper half hands its to the lower, and again
#pragma unroll
  for (int nr = 0; nr < NR; ++nr) l_run[nr] = xor_sum(l_run[nr]);
#pragma unroll
  for (int step = NW / 2; step >= 1; step >>= 1) {
    if (2 * step > wph) continue;
    // a head's waves hand over in a part of the LDS of their own
    const int from = E2M1 ? wave / wph * (wph / 2) : 0;
    __syncthreads();
    if (lane_wave >= step && lane_wave < 2 * step) {
      const int w = from + lane_wave - step;
#pragma unroll
      for (int nr = 0; nr < NR; ++nr) {
        const int r = 16 * nr + col;
        if (q4 == 0) {
          sh_m[w][r] = m_run[nr];
          sh_l[w][r] = l_run[nr];
        }
        float *row = sh.o + (w * kRows + r) * F::kPad;
#pragma unroll
        for (int t = 0; t < F::kTiles; ++t) *(f32x4 *)(row + t * 16 + q4 * 4) = acc[nr][t];
      }
    }
    __syncthreads();
    if (lane_wave < step) {
      const int w = from + lane_wave;
#pragma unroll
      for (int nr = 0; nr < NR; ++nr) {
        const int r = 16 * nr + col;
        const float mo = sh_m[w][r], lo2 = sh_l[w][r];
        const float m_new = fmaxf(m_run[nr], mo);
        const float x = m_new == -INFINITY ? 1.0f : fast_exp2(m_run[nr] - m_new);
        const float y = m_new == -INFINITY ? 1.0f : fast_exp2(mo - m_new);
        m_run[nr] = m_new;
        l_run[nr] = l_run[nr] * x + lo2 * y;
        const float *row = sh.o + (w * kRows + r) * F::kPad;
#pragma unroll
        for (int t = 0; t < F::kTiles; ++t) acc[nr][t] = acc[nr][t] * x + *(const f32x4 *)(row + t * 16 + q4 * 4) * y;
      }
    }
  }
  if (lane_wave == 0) {
  if (sh_odd) {
    // p is above 0 wherever a row sees a slot: an infinity or NaN in it is the sum
    uint64_t some = 0;           // kBoth: of 64 slots those with a block past the finite powers
    for (int j = c0; j < c1; ++j) {
      if constexpr (kBoth) {
        if (((j - c0) & (kWave - 1)) == 0) {
          const SlotPlace pl = j + lane < c1 ? slot_place(a.c, trow, (uint32_t)(j + lane)) : SlotPlace{-1, 0};
          const uint8_t *powers = a.c.v_power + (uint64_t)place_number(a.c, pl, h) * (D / kPowerBlock);
          bool has = false;
          for (int b = 0; b < D / kPowerBlock; ++b) has |= powers[b] > T::kE2m1Top;
          some = __ballot(has && pl.page >= 0);
        }
        if (!((some >> ((j - c0) & (kWave - 1))) & 1u)) continue;
      } else if (!(j > sp.first || (a.window > 0 && j <= last_pos - a.window))) {
        continue;
      }
      const SlotPlace pl = slot_place(a.c, trow, (uint32_t)j);
      const int64_t o = place_offset(a.c, pl);
      if (o < 0) continue;
      const uint8_t *powers = E2M1 ? a.c.v_power + (uint64_t)place_number(a.c, pl, h) * (D / kPowerBlock) : nullptr;
#pragma unroll
      for (int nr = 0; nr < NR; ++nr) {
        if (j > pos[nr] || (a.window > 0 && j <= pos[nr] - a.window)) continue;
        int t0 = 0, base = 0;
#pragma unroll
        for (int n = 0; n < VPieces<D>::n; ++n) {
          const int w = VPieces<D>::w[n];
#pragma unroll
          for (int rg = 0; rg < 4; ++rg)
#pragma unroll
            for (int t = 0; t < w; t += 2) {
              const int d = base + (q4 * 4 + rg) * w + t;
              const char *e = vbase + o + (E2M1 ? d / 2 : d * F::kBytes);
              const uint32_t x = E2M1 ? T::template from_e2m1<0>(*(const uint8_t *)e, powers[d / kPowerBlock])
                               : E4M3 ? T::template from_e4m3<false>(*(const uint16_t *)e) : *(const uint32_t *)e;
              acc[nr][t0 + t][rg] += nonfinite_lo<T>(x);
              acc[nr][t0 + t + 1][rg] += nonfinite_hi<T>(x);
            }
          t0 += w;
          base += 16 * w;
        }
      }
    }
  }
  const float vs = E4M3 ? a.c.v_scale[h] : 1.0f;
#pragma unroll
  for (int nr = 0; nr < NR; ++nr) {
    const int r = 16 * nr + col;
    if (r >= R) continue;
    const int tok = (int)fast_div(a.gdiv, (uint32_t)r), g = r - tok * G;
    const int64_t at = (sp.t0 + tok) * heads + h * G + g;
    const float l = l_run[nr];
    float *po = nullptr;
    char *out = nullptr;
    float mul = vs;
    if (part) {
      if (q4 == 0) a.part_ml[part_at + r] = make_float2(m_run[nr], l);
      po = a.part_o + (part_at + r) * D;
      if (!(l > 0.0f || l != l)) continue;      // nothing here: the join skips it
    } else {
      if (q4 == 0) a.lse[at] = l > 0.0f || l != l ? (m_run[nr] + __log2f(l)) * kLn2 : -INFINITY;
      mul = l > 0.0f || l != l ? vs / l : 0.0f;
      out = a.out + at * D * 2;
    }
    // accumulator register rg of column tile t: column base + (4 q4 + rg) w + t
    int ct = 0, base = 0;
#pragma unroll
    for (int n = 0; n < VPieces<D>::n; ++n) {
      const int w = VPieces<D>::w[n];
#pragma unroll
      for (int rg = 0; rg < 4; ++rg) {
        const int d = base + (q4 * 4 + rg) * w;
#pragma unroll
        for (int t = 0; t < w; t += 2) {
          const float x = acc[nr][ct + t][rg] * mul, y = acc[nr][ct + t + 1][rg] * mul;
          if (po) *(f32x2 *)(po + d + t) = (f32x2){x, y};
          else *(uint32_t *)(out + (d + t) * 2) = T::pack(x, y);
        }
      }
      ct += w;
      base += 16 * w;
    }
  }
  }      // the first wave
  left -= (uint32_t)(t1 - t0);
  if (a.whole || left == 0) return;
  t0 = 0;
  if (E2M1 || ++h == H) {
    if (!E2M1) h = 0;
    if (++s >= a.c.seqs) return;
    span = few_span(a, s);
  }
  __syncthreads();             // the next piece writes the same LDS
  }
}

// A part's place: a work-group's run starts a longer row of parts in its second one.
__device__ __forceinline__ int64_t part_slot(const AttendArgs &a, int w, int w0, int h, int rows) {
  const int64_t wg = a.by_head ? (int64_t)w * a.c.heads + h : w;
  return (wg * 2 + (w == w0 ? 1 : 0)) * rows;
}

// Weights from kept scores: a thread adds up the rows' 2^(score - lse) for four slots in a row.
// 25 bytes a slot at four rows: the chain of loads before the sum costs more than they do, so a
// work-group takes many slots.  lse comes from the parts, so that nothing waits for their join.
constexpr int kScoreGroups = 2, kScoreAhead = 4;      // groups of a thread; rows loaded before lse is known
static_assert(kScoreSlots == 4 * kScoreGroups * kFinishThreads, "four slots a group");
__device__ __forceinline__ void score_sums(const AttendArgs &a, int block, int part_rows, float *lse2) {
  const int H = a.c.heads, G = a.group, tid = threadIdx.x;
  const int blocks = (a.max_len + kScoreSlots - 1) / kScoreSlots;
  const int sh = block / blocks, s = sh / H, h = sh - s * H;
  const FewSpan span = few_span(a, s);
  const SeqSpan &sp = span.sp;
  const int j0 = (block - sh * blocks) * kScoreSlots;
  const int R = sp.m * G;
  if (j0 >= sp.n) return;
  // four slots share a page, and their weights 16 bytes, where the page size allows
  const bool together = a.c.page.d % 4 == 0;
  const int lo = a.window > 0 && sp.first - a.window + 1 > 0 ? sp.first - a.window + 1 : 0;
  const int32_t *trow = a.c.table + (int64_t)s * a.c.table_stride;
  SlotPlace pl[kScoreGroups][4];
  f32x4 ahead[kScoreGroups][kScoreAhead];
  const float *z[kScoreGroups];
  bool seen[kScoreGroups];
#pragma unroll
  for (int g = 0; g < kScoreGroups; ++g) {
    const int j = j0 + 4 * (g * kFinishThreads + tid);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      pl[g][u] = SlotPlace{-1, 0};
      if (j + u < sp.n && (u == 0 || !together)) pl[g][u] = slot_place(a.c, trow, (uint32_t)(j + u));
    }
    // scores exist from the tile of `lo` to the group of four of `hi`
    seen[g] = j + 3 >= lo && j < span.hi;
    z[g] = a.scores + ((int64_t)sh * (a.score_stride / 4) + (j >> 2)) * a.score_rows * 4;
#pragma unroll
    for (int r = 0; r < kScoreAhead; ++r)
      ahead[g][r] = seen[g] && r < R ? *(const f32x4 *)(z[g] + r * 4) : (f32x4){0, 0, 0, 0};
  }
  int w0 = 0, w1 = 0;
  if (!a.whole && R > 0) part_range(a, a.line[a.c.seqs], a.line[s], h, span.tiles, &w0, &w1);
  // the rows' lse: `width` lanes a row, each every width-th part in order, then the lanes two by two
  const int width = R <= 4 ? 64 : (R <= 8 ? 32 : (R <= 16 ? 16 : 8)), r = tid / width;
  static_assert(kFinishThreads / 8 >= kFewRowsMax, "every row has its lanes");
  float l2 = -INFINITY;
  if (w0 == w1) {
    const int tok = (int)fast_div(a.gdiv, r), g = r - tok * G;
    if (r < R) l2 = a.lse[(sp.t0 + tok) * ((int64_t)H * G) + h * G + g] * kLog2e;
  } else {
    float top = -INFINITY, l = 0.0f;
    const auto add = [&](float m, float y) {
      if (!(y > 0.0f || y != y)) return;
      const float m_new = fmaxf(top, m);
      l = l * fast_exp2(top - m_new) + y * fast_exp2(m - m_new);
      top = m_new;
    };
    if (r < R) {
#pragma unroll 4
      for (int w = w0 + (tid & (width - 1)); w <= w1; w += width) {
        const float2 x = a.part_ml[part_slot(a, w, w0, h, part_rows) + r];
        add(x.x, x.y);
      }
    }
    for (int o = 1; o < width; o <<= 1) add(__shfl_xor(top, o), __shfl_xor(l, o));
    l2 = l > 0.0f || l != l ? top + __log2f(l) : -INFINITY;
  }
  if (r < R && (tid & (width - 1)) == 0) lse2[r] = l2 == -INFINITY ? INFINITY : l2;   // a row that sees nothing gives 0
  __syncthreads();
#pragma unroll
  for (int g = 0; g < kScoreGroups; ++g) {
    const int j = j0 + 4 * (g * kFinishThreads + tid);
    if (j >= sp.n) break;
    f32x4 w = (f32x4){0, 0, 0, 0};
    const auto add = [&](f32x4 x, float l) {
#pragma unroll
      for (int u = 0; u < 4; ++u) w[u] += x[u] == -INFINITY ? 0.0f : fast_exp2(x[u] - l);
    };
    if (seen[g]) {
#pragma unroll
      for (int r = 0; r < kScoreAhead; ++r)
        if (r < R) add(ahead[g][r], lse2[r]);
#pragma unroll 4
      for (int r = kScoreAhead; r < R; ++r) add(*(const f32x4 *)(z[g] + r * 4), lse2[r]);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) w[u] = j + u >= lo && j + u < span.hi ? w[u] : 0.0f;
    if (together && j + 3 < sp.n) {
      if (pl[g][0].page < 0) continue;
      f32x4 *at = (f32x4 *)(a.c.weights + ((int64_t)pl[g][0].page * H + h) * a.c.page.d + pl[g][0].row);
      if (a.decay != 0.0f) w += a.decay * *at;
      *at = w;
      continue;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const SlotPlace p = together ? SlotPlace{pl[g][0].page, pl[g][0].row + u} : pl[g][u];
      if (j + u >= sp.n || p.page < 0) continue;
      float *at = a.c.weights + ((int64_t)p.page * H + h) * a.c.page.d + p.row;
      *at = a.decay != 0.0f ? a.decay * *at + w[u] : w[u];
    }
  }
}

// The second pass of the few-rows form: work-groups below `joins` join the parts of a (sequence,
// head), `rows_per` rows each, `slices` of them a row's columns; the others turn kept scores into weights.
//   out = sum_k 2^(m_k - M) o_k / sum_k 2^(m_k - M) l_k
// over the work-groups k of the run, under a running maximum M, in order within each of the groups
// of dim / 4 threads, then the groups in order.
template <class T, int D, int NR>
__global__ __launch_bounds__(kFinishThreads) void finish_few_kernel(AttendArgs a, int joins, int rows_per, int slices) {
  const int lanes = D / 4 / slices, groups = kFinishThreads / lanes;      // threads of a group, a float4 each
  __shared__ f32x4 part[kFinishThreads];
  __shared__ float2 part_ml[kFinishThreads];
  __shared__ float lse2[kFewRowsMax];
  if ((int)blockIdx.x >= joins) return score_sums(a, blockIdx.x - joins, 16 * NR, lse2);
  const int H = a.c.heads, G = a.group, tid = threadIdx.x;
  const int64_t heads = (int64_t)H * G;
  const int blocks = (a.max_q * G + rows_per - 1) / rows_per;
  const int block = blockIdx.x / slices, slice = blockIdx.x - block * slices;
  const int sh = block / blocks, s = sh / H, h = sh - s * H;
  const uint32_t share = a.line[a.c.seqs], begin = a.line[s];     // on their way with the lengths
  const FewSpan span = few_span(a, s);
  const int R = span.sp.m * G;
  if (R == 0) return;
  int w0, w1;
  part_range(a, share, begin, h, span.tiles, &w0, &w1);
  if (w0 == w1) return;        // one work-group had all of it
  // a row by per_row groups of threads
  const int g = tid / lanes, d4 = tid - g * lanes + slice * lanes;
  const int per_row = groups / rows_per, gr = g / per_row, gk = g - gr * per_row;
  const int r = (block - sh * blocks) * rows_per + gr;
  const bool mine = gr < rows_per && r < R;
  f32x4 acc = (f32x4){0, 0, 0, 0};
  float l = 0.0f, top = -INFINITY;
  const auto add = [&](float m, float y, f32x4 o) {
    if (!(y > 0.0f || y != y)) return;         // a part without a slot: its sums were not written
    const float m_new = fmaxf(top, m), x = fast_exp2(top - m_new), z = fast_exp2(m - m_new);
    l = l * x + y * z;
    acc = acc * x + o * z;
    top = m_new;
  };
  if (mine) {
    // eight parts are loaded before the first is added
    for (int w = w0 + gk; w <= w1; w += 8 * per_row) {
      float2 x[8];
      f32x4 o[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int v = w + u * per_row <= w1 ? w + u * per_row : w1;
        const int64_t at = part_slot(a, v, w0, h, 16 * NR) + r;
        x[u] = a.part_ml[at];
        o[u] = *(const f32x4 *)(a.part_o + at * D + d4 * 4);
      }
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (w + u * per_row <= w1) add(x[u].x, x[u].y, o[u]);
    }
  }
  part[tid] = acc;
  part_ml[tid] = make_float2(top, l);
  __syncthreads();
  if (!mine || gk != 0) return;
  for (int k = 1; k < per_row; ++k) add(part_ml[tid + k * lanes].x, part_ml[tid + k * lanes].y, part[tid + k * lanes]);
  const int tok = (int)fast_div(a.gdiv, (uint32_t)r);
  const int64_t row = (span.sp.t0 + tok) * heads + h * G + (r - tok * G);
  const bool any = l > 0.0f || l != l;
  const float mul = any ? 1.0f / l : 0.0f;
  if (d4 == 0) a.lse[row] = any ? (top + __log2f(l)) * kLn2 : -INFINITY;
  const f32x4 o = any ? acc * mul : (f32x4){0, 0, 0, 0};
  *(u32x2 *)(a.out + (row * D + d4 * 4) * 2) = (u32x2){T::pack(o[0], o[1]), T::pack(o[2], o[3])};
}

// One (type, cache, dim) of the few-rows form.  Returns the work-groups that fit the device at
// once when `grid` is 0.
template <class T, int BITS, int D, int NR, bool SCORES>
int few_variant(const AttendArgs &a, int grid, int join_rows, hipStream_t st) {
  if (grid == 0) {
    static std::atomic<int> fit{0};
    int n = fit.load(std::memory_order_relaxed);
    if (n <= 0) {
      if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&n, (const void *)attend_few_kernel<T, BITS, D, NR, SCORES, kFewWaves, false>,
                                                       kFewThreads, 0) != hipSuccess || n < 1)
        return -1;
      fit.store(n, std::memory_order_relaxed);
    }
    return n;
  }
  if constexpr (NR == 1 && D <= 128) {
    if (a.whole == 2) attend_few_kernel<T, BITS, D, NR, SCORES, 8, false><<<dim3((unsigned)grid), 8 * kWave, 0, st>>>(a);
  }
  if (a.far)
    attend_few_kernel<T, BITS, D, NR, SCORES, kFewWaves, true><<<dim3((unsigned)grid), kFewThreads, 0, st>>>(a);
  else if (!(NR == 1 && D <= 128 && a.whole == 2))
    attend_few_kernel<T, BITS, D, NR, SCORES, kFewWaves, false><<<dim3((unsigned)grid), kFewThreads, 0, st>>>(a);
  const int64_t sh = (int64_t)a.c.seqs * a.c.heads;
  const int64_t joins = join_rows > 0 ? ((int64_t)a.max_q * a.group + join_rows - 1) / join_rows * sh * a.join_slices : 0;
  const int64_t sums = SCORES ? (a.max_len + kScoreSlots - 1) / kScoreSlots * sh : 0;
  if (joins + sums > 0)
    finish_few_kernel<T, D, NR><<<dim3((unsigned)(joins + sums)), kFinishThreads, 0, st>>>(a, (int)joins, join_rows, a.join_slices);
  return 0;
}
template <class T, int BITS, int D>
int launch_few_dim(const AttendArgs &a, int row_tiles, int grid, int join_rows, hipStream_t st) {
  if (row_tiles == 1)
    return a.score_stride ? few_variant<T, BITS, D, 1, true>(a, grid, join_rows, st)
                          : few_variant<T, BITS, D, 1, false>(a, grid, join_rows, st);
  return a.score_stride ? few_variant<T, BITS, D, 2, true>(a, grid, join_rows, st)
                        : few_variant<T, BITS, D, 2, false>(a, grid, join_rows, st);
}

template <class T, int BITS>
int launch_few(const AttendArgs &a, int dim, int row_tiles, int grid, int join_rows, hipStream_t st) {
  if (dim == 64) return launch_few_dim<T, BITS, 64>(a, row_tiles, grid, join_rows, st);
  if (dim == 96) return launch_few_dim<T, BITS, 96>(a, row_tiles, grid, join_rows, st);
  if (dim == 128) return launch_few_dim<T, BITS, 128>(a, row_tiles, grid, join_rows, st);
  return launch_few_dim<T, BITS, 256>(a, row_tiles, grid, join_rows, st);
}

}  // namespace kmi
