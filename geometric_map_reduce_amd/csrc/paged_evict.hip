// paged_evict.hip -- eviction from a paged cache by attention weight.
//
// Of a sequence's slots that are there each key/value head keeps `budget`: those among the
// first `sink`, those among the last `recent`, and of the others the ones with the largest weights
// (equal weights: the lower slot).  Kept slots move, in their order, to slots 0 .. of the pages in
// new_table, keys, values and weights alike; where no more than `budget` are there, all of them.
// A slot of a page that is not there is left out: a row kept for it would be one that nothing writes
// and every later query sees.  (Pages are the same for all heads, so the heads keep equally many.)
//
// Selection: one work-group per (sequence, head) holds up to 32,768 weights in LDS as whole numbers of
// the same order (longer rows are read again for each pass) and finds the smallest kept one by up to
// three passes over 11, 11 and 10 bits, with counts in LDS (whole numbers, so the order of the additions
// does not matter).  Once no more than 64 keys share the digits found, they are ranked by weight and
// slot instead.  In the end a thread has up to 32 slots in a row and writes down its own; their places
// come from a scan of the threads' counts.
// Loading, a thread has four slots in a row: one page number and one 16-byte load where pages are whole
// aligned quadruples, slot by slot otherwise.  64 rows of up to 32,768 slots take 22 us (9 for the loads
// and the first pass, on 64 compute units), 32 rows of 1,025 slots 9.5 us; instructions bound the long rows,
// latency the short ones.  0.6 to 1 us of either is the look through the table for pages that are not there.
// 256 keys of a wave that all meet one count add to it once (cleared weights are
// all equal).  Slot by slot loads and keys in registers under unrolled loops took 43 us, 16-byte loads 32,
// keys in LDS 30 (the last round by ballots over the waves).  The move is a second kernel, one 16-byte
// piece of a key and of a value row per thread, bound by HBM: 268 MB read and written in 49 us.
#include "paged.h"

namespace kmi {
namespace {

constexpr int kSelectWaves = kSelectThreads / kWave;
constexpr int kBins = 2048;             // counts of a pass
constexpr int kHistCopies = 2;          // even and odd lanes: fewer collisions
constexpr int kHistStride = kBins + 32; // a bin's copies lie in different banks
constexpr int kQuad = 4;                // slots in a row of a thread
constexpr int kGroup = kQuad * kSelectThreads;
constexpr int kGroupsFew = 1, kGroupsMost = 8;   // groups of keys in LDS: 16 and 128 KB

// Whole numbers ordered as the floats are; -0 equals 0, NaN above everything but kForced.
constexpr uint32_t kAbsent = 1u, kForced = 0xffffffffu;      // below and above the keys of all weights
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return kForced - 1;
  const uint32_t b = __float_as_uint(w == 0.0f ? 0.0f : w);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// Where a quadruple of keys lies in LDS: threads that read a group, one quadruple each, and threads that read
// eight in a row both meet all banks.
__device__ __forceinline__ int quad_at(int q) { return q ^ ((q >> 4) & 7); }

template <int kGroups>
struct SelectShared {
  u32x4 key[kGroups * kSelectThreads];
  __align__(16) uint32_t hist[kHistStride * kHistCopies];
  __align__(16) uint32_t wave_sum[kSelectWaves];
  uint32_t prefix, need, count;
  uint32_t cand_key[kWave], cand_slot[kWave], cand_rank[kWave], cands;
  uint32_t cut_key, cut_slot;
};

// Sum of the waves before this one; all of them in `total`.
__device__ __forceinline__ uint32_t before_wave(const uint32_t *wave_sum, int wave, uint32_t *total) {
  uint32_t before = 0, all = 0;
#pragma unroll
  for (int w4 = 0; w4 < kSelectWaves / 4; ++w4) {
    const u32x4 x = ((const u32x4 *)wave_sum)[w4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      before += w4 * 4 + u < wave ? x[u] : 0u;
      all += x[u];
    }
  }
  *total = all;
  return before;
}
template <int kGroups>
__global__ __launch_bounds__(kSelectThreads) void select_kernel(EvictArgs a) {
  constexpr int kSegment = kGroups * kGroup, kBatch = kGroups < 4 ? kGroups : 4;
  __shared__ SelectShared<kGroups> sh;
  const int H = a.c.heads;
  const int s = blockIdx.x / H, h = blockIdx.x - s * H;
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  int64_t n64 = a.c.lens[s];
  const int64_t most = (int64_t)a.c.table_width * a.c.page.d;
  n64 = n64 < 0 ? 0 : (n64 > most ? most : n64);
  const int n = (int)n64;
  int32_t *kept = a.kept + ((int64_t)s * H + h) * a.budget;
  const int32_t *trow = a.c.table + (int64_t)s * a.c.table_stride;
  const uint32_t ps = a.c.page.d;
  // slots of pages that are not there: they are left out, whatever their place
  uint32_t lost = 0;
  for (int64_t j = (int64_t)tid * ps; j < n; j += (int64_t)kSelectThreads * ps)
    if ((uint32_t)trow[fast_div(a.c.page, (uint32_t)j)] >= a.c.pages) lost += n - j < (int64_t)ps ? (uint32_t)(n - j) : ps;
  const uint32_t lost_upto = wave_scan_u32(lost);
  if (lane == kWave - 1) sh.wave_sum[wave] = lost_upto;
  __syncthreads();
  uint32_t absent;
  before_wave(sh.wave_sum, 0, &absent);
  absent = __builtin_amdgcn_readfirstlane(absent);
  const bool holes = absent != 0;
  const int keep = n - (int)absent < a.budget ? n - (int)absent : a.budget;
  if (h == 0 && tid == 0) a.new_lens[s] = keep;
  if (!holes && n <= a.budget) {
    for (int r = tid; r < a.budget; r += kSelectThreads) kept[r] = r < n ? r : -1;
    return;
  }
  // with holes the first and the last slots are chosen like the others, by a key above all weights'
  const int sink = holes ? 0 : a.sink, recent = holes ? 0 : a.recent, need0 = keep - sink - recent;
  for (int r = tid; r < sink; r += kSelectThreads) kept[r] = r;
  for (int r = tid; r < recent; r += kSelectThreads) kept[a.budget - recent + r] = n - recent + r;
  for (int r = keep + tid; r < a.budget; r += kSelectThreads) kept[r] = -1;
  if (need0 == 0) return;
  // the slots in question, counted from `base0`: skip .. M - 1
  const int base0 = sink / kQuad * kQuad, skip = sink - base0, M = n - recent - base0;
  const int segments = (M + kSegment - 1) / kSegment;
  // groups of a segment that hold any, in whole batches: a batch's keys leave LDS together
  const auto groups_of = [&](int from) {
    const int left = (M - from + kBatch * kGroup - 1) / (kBatch * kGroup) * kBatch;
    return left < kGroups ? left : kGroups;
  };
  const auto quads = [&](int g, u32x4 (&k)[kBatch]) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) k[u] = sh.key[quad_at((g + u) * kSelectThreads + tid)];
  };
  // Keys of a segment to LDS, each thread its own quadruples.  An absent slot's is below every weight's, and
  // that of a place outside skip .. M is 0: it is never among the largest that there are.
  const auto put = [&](int g, int i, u32x4 k) {      // slots i .. of group g
    if (holes) {                                     // base0 is 0
#pragma unroll
      for (int e = 0; e < kQuad; ++e)
        if (k[e] != kAbsent && (i + e < a.sink || i + e >= n - a.recent)) k[e] = kForced;
    }
#pragma unroll
    for (int e = 0; e < kQuad; ++e) k[e] = i + e >= skip && i + e < M ? k[e] : 0u;
    sh.key[quad_at(g * kSelectThreads + tid)] = k;
  };
  const bool whole = ps % kQuad == 0 && ((uintptr_t)a.c.weights & 15) == 0;   // a quadruple in one page, aligned
  const auto load = [&](int from) {
    const int groups = groups_of(from);
    if (whole) {
      // page and row go on by a group's slots with an addition each
      const uint32_t j0 = (uint32_t)(base0 + from + tid * kQuad), step_page = kGroup / ps, step_row = kGroup - step_page * ps;
      uint32_t pi = fast_div(a.c.page, j0), row = j0 - pi * ps, page[kGroups], rows = row;
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        int32_t pg = -1;
        if (pi < a.c.table_width && from + g * kGroup + tid * kQuad < M) pg = trow[pi];
        page[g] = (uint32_t)pg;
        pi += step_page;
        row += step_row;
        if (row >= ps) { row -= ps; ++pi; }
      }
      f32x4 w[kGroups];
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        w[g] = (f32x4){0, 0, 0, 0};
        // its number is below 2^32: the caller sees to it
        if (page[g] < a.c.pages) w[g] = *(const f32x4 *)(a.c.weights + ((page[g] * (uint32_t)H + (uint32_t)h) * ps + rows));
        rows += step_row;
        if (rows >= ps) rows -= ps;
      }
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        if (g >= groups) break;
        u32x4 k = (u32x4){kAbsent, kAbsent, kAbsent, kAbsent};
        if (page[g] < a.c.pages)
          k = (u32x4){weight_key(w[g][0]), weight_key(w[g][1]), weight_key(w[g][2]), weight_key(w[g][3])};
        put(g, from + g * kGroup + tid * kQuad, k);
      }
      return;
    }
#pragma unroll 2
    for (int g = 0; g < groups; ++g) {
      u32x4 k = (u32x4){kAbsent, kAbsent, kAbsent, kAbsent};
#pragma unroll
      for (int e = 0; e < kQuad; ++e) {
        const int i = from + g * kGroup + tid * kQuad + e;
        if (i >= M) continue;
        const SlotPlace p = slot_place(a.c, trow, (uint32_t)(base0 + i));
        if (p.page >= 0) k[e] = weight_key(a.c.weights[((uint32_t)p.page * (uint32_t)H + (uint32_t)h) * ps + p.row]);
      }
      put(g, from + g * kGroup + tid * kQuad, k);
    }
  };

  // the need-th largest key, digit by digit
  uint32_t prefix = 0, need = (uint32_t)need0, count = 0, cut = 0xffffffffu;
  if (tid == 0) sh.cands = 0;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), bits = pass == 2 ? 10 : 11;
    for (int i = tid; i < kHistStride * kHistCopies / 4; i += kSelectThreads) ((u32x4 *)sh.hist)[i] = (u32x4){0, 0, 0, 0};
    __syncthreads();
    uint32_t *mine = sh.hist + (lane & (kHistCopies - 1)) * kHistStride;
#pragma unroll 1
    for (int from = 0; from < M; from += kSegment) {
      if (pass == 0 || segments > 1) load(from);
      const int groups = groups_of(from);
#pragma unroll 1
      for (int g0 = 0; g0 < groups; g0 += kBatch) {
        u32x4 k[kBatch];
        quads(g0, k);
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          uint32_t bin[kQuad];
          bool in[kQuad], same = true;
#pragma unroll
          for (int e = 0; e < kQuad; ++e) {
            in[e] = pass == 0 || (k[u][e] >> (shift + bits)) == (prefix >> (shift + bits));
            bin[e] = (k[u][e] >> shift) & ((1u << bits) - 1u);
            same &= in[e] && bin[e] == (uint32_t)__builtin_amdgcn_readfirstlane(bin[0]);
          }
          if (__all(same)) {
            if (lane == 0) atomicAdd(&mine[bin[0]], (uint32_t)(kQuad * kWave));
            continue;
          }
#pragma unroll
          for (int e = 0; e < kQuad; ++e)
            if (in[e]) atomicAdd(&mine[bin[e]], 1u);
        }
      }
    }
    __syncthreads();
    // thread t has the counts 2 t and 2 t + 1 from the top
    const int low = kBins - 2 - 2 * tid;
    uint32_t cnt[2] = {0, 0};
#pragma unroll
    for (int c = 0; c < kHistCopies; ++c) {
      const u32x2 x = *(const u32x2 *)&sh.hist[c * kHistStride + low];
      cnt[0] += x.y;
      cnt[1] += x.x;
    }
    const uint32_t own = cnt[0] + cnt[1], upto = wave_scan_u32(own);
    if (lane == kWave - 1) sh.wave_sum[wave] = upto;
    __syncthreads();
    uint32_t total;
    uint32_t above = upto - own + before_wave(sh.wave_sum, wave, &total);
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      if (above < need && need <= above + cnt[b]) {
        sh.prefix = prefix | ((uint32_t)(kBins - 1 - (2 * tid + b)) << shift);
        sh.need = need - above;
        sh.count = cnt[b];
      }
      above += cnt[b];
    }
    __syncthreads();
    prefix = sh.prefix;
    need = sh.need;
    count = sh.count;
    if (count == need) break;          // all that share the digits so far are kept
    if (count <= kWave && segments == 1) {
      // few share them: they are ranked by weight and slot, each wave against a part of them
      const int groups = groups_of(0);
#pragma unroll 1
      for (int g0 = 0; g0 < groups; g0 += kBatch) {
        u32x4 k[kBatch];
        quads(g0, k);
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          const int i = (g0 + u) * kGroup + tid * kQuad;
#pragma unroll
          for (int e = 0; e < kQuad; ++e) {
            if ((k[u][e] >> shift) == (prefix >> shift)) {
              const uint32_t at = atomicAdd(&sh.cands, 1u);
              sh.cand_key[at] = k[u][e];
              sh.cand_slot[at] = (uint32_t)(i + e);
            }
          }
        }
      }
      if (tid < kWave) sh.cand_rank[tid] = 0;
      __syncthreads();
      const uint32_t k = sh.cand_key[lane], i = sh.cand_slot[lane];
      uint32_t before = 0;
      for (uint32_t m = wave; m < count; m += kSelectWaves) {
        const uint32_t km = __builtin_amdgcn_readlane(k, m), im = __builtin_amdgcn_readlane(i, m);
        before += km > k || (km == k && im < i);
      }
      if (before) atomicAdd(&sh.cand_rank[lane], before);
      __syncthreads();
      if (tid < (int)count && sh.cand_rank[tid] == need - 1) {
        sh.cut_key = k;
        sh.cut_slot = i;
      }
      __syncthreads();
      prefix = sh.cut_key;
      cut = sh.cut_slot;
      need = count;                    // settled
      break;
    }
  }
  // kept: keys above `prefix`, and those equal to it up to slot `cut`.  Without a cut yet and with
  // more equal keys than wanted, a first round over the equal ones finds the need-th.  In either
  // round a slot's place is the number of slots before it: counts of the threads, scanned.
#pragma unroll 1
  for (int round = need == count ? 1 : 0; round < 2; ++round) {
    uint32_t base = 0;
#pragma unroll 1
    for (int from = 0; from < M; from += kSegment) {
      if (segments > 1) load(from);
      // here a thread has `groups` quadruples in a row, 32 slots at most
      const int groups = groups_of(from), first = tid * groups;
      if (segments > 1) __syncthreads();
      uint32_t mine = 0;               // its slots as bits
      for (int g = 0; g < groups; ++g) {
        const u32x4 k = sh.key[quad_at(first + g)];
        const int i = from + (first + g) * kQuad;
#pragma unroll
        for (int e = 0; e < kQuad; ++e) {
          const bool eq = k[e] == prefix;
          const bool in = round == 0 ? eq : k[e] > prefix || (eq && (uint32_t)(i + e) <= cut);
          mine |= (in ? 1u << e : 0u) << (g * kQuad);
        }
      }
      const uint32_t own = (uint32_t)__popc(mine);
      uint32_t total;
      const uint32_t upto = wave_scan_u32(own);
      if (lane == kWave - 1) sh.wave_sum[wave] = upto;
      __syncthreads();
      uint32_t place = base + upto - own + before_wave(sh.wave_sum, wave, &total);
      for (; mine; mine &= mine - 1, ++place) {
        const int i = from + first * kQuad + __ffs(mine) - 1;
        if (round == 1) kept[sink + place] = base0 + i;
        else if (place == need - 1) sh.cut_slot = (uint32_t)i;
      }
      base += total;
      __syncthreads();
    }
    if (round == 0) cut = sh.cut_slot;
  }
}

// One thread per 16-byte piece of a kept slot's key row, and the same piece of its value row.  FAR: loads
// that pass the caches by, where more is moved than the last level holds (551 MB read and written: 135 us
// a call by way of it, 113 past it; 277 MB 70 and 69, 138 MB 45 and 48).
template <bool FAR>
__global__ __launch_bounds__(256) void move_kernel(EvictArgs a, int pieces, int64_t total) {
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (id >= total) return;
  const int64_t row = id / pieces;
  const int piece = (int)(id - row * pieces);
  const int32_t src = a.kept[row];
  if (src < 0) return;
  const int64_t sh = row / a.budget;
  const int r = (int)(row - sh * a.budget);
  const int s = (int)(sh / a.c.heads), h = (int)(sh - (int64_t)s * a.c.heads);
  const SlotPlace from = slot_place(a.c, a.c.table + (int64_t)s * a.c.table_stride, (uint32_t)src);
  const uint32_t pi = fast_div(a.c.page, (uint32_t)r);
  int32_t pg = -1;
  if (pi < a.new_width) pg = a.new_table[(int64_t)s * a.new_stride + pi];
  if (from.page < 0 || (uint32_t)pg >= a.c.pages) return;
  const SlotPlace to{pg, (uint32_t)r - pi * a.c.page.d};
  const int64_t head = (int64_t)h * a.c.head_stride + (int64_t)piece * 16;
  const int64_t fo = place_offset(a.c, from) + head, dst = place_offset(a.c, to) + head;
  const u32x4 k = load_once<u32x4, FAR>(a.c.k + fo);
  const u32x4 v = load_once<u32x4, FAR>(a.c.v + fo);
  *(u32x4 *)(a.c.k + dst) = k;
  *(u32x4 *)(a.c.v + dst) = v;
  if (piece == 0)
    a.c.weights[((int64_t)to.page * a.c.heads + h) * a.c.page.d + to.row] =
        a.c.weights[((int64_t)from.page * a.c.heads + h) * a.c.page.d + from.row];
}

}  // namespace

void launch_evict(const EvictArgs &a, hipStream_t st) {
  const dim3 grid((unsigned)(a.c.seqs * a.c.heads));
  if ((int64_t)a.c.table_width * a.c.page.d <= kGroupsFew * kGroup)
    select_kernel<kGroupsFew><<<grid, kSelectThreads, 0, st>>>(a);
  else
    select_kernel<kGroupsMost><<<grid, kSelectThreads, 0, st>>>(a);
  const int pieces = a.c.dim * a.itemsize / 16;
  const int64_t total = (int64_t)a.c.seqs * a.c.heads * a.budget * pieces;
  const dim3 move((unsigned)((total + 255) / 256));
  if (64.0 * (double)total > kLastLevel) move_kernel<true><<<move, 256, 0, st>>>(a, pieces, total);
  else move_kernel<false><<<move, 256, 0, st>>>(a, pieces, total);
}

}  // namespace kmi
