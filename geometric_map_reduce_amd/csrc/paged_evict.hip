// paged_evict.hip -- eviction from a paged cache by attention weight.
//
// Of a sequence's n slots each key/value head keeps `budget`: the first `sink`, the last
// `recent`, and of those between the ones with the largest weights (equal weights: the lower
// slot).  Kept slots move, in their order, to slots 0 .. of the pages in new_table, keys,
// values and weights alike; n <= budget keeps them all.
//
// Selection: one work-group per (sequence, head) holds up to 32,768 weights in registers as whole
// numbers of the same order (longer rows are read again for each pass), finds the smallest kept one
// by three passes over 11, 11 and 10 bits (counts in LDS: whole numbers, so the order of the
// additions does not matter), and gives every slot its place from the counts of the waves before
// it.  It is bound by the latency of its steps: page numbers and weights are loaded eight at a
// time, lanes count in eight copies, and a wave whose lanes all meet one count adds to it once
// (cleared weights are all equal).  The move is a second kernel, one 16-byte piece of a key and of
// a value row per thread, bound by HBM.
#include "paged.h"

namespace kmi {
namespace {

constexpr int kSelectThreads = 1024;
constexpr int kSelectWaves = kSelectThreads / kWave;
constexpr int kBins = 2048;             // counts of a pass
constexpr int kHistCopies = 8;          // lanes of a wave spread over copies: fewer collisions
constexpr int kHeld = 32;               // keys of a thread
constexpr int kBatch = 8;
constexpr int kSegment = kHeld * kSelectThreads;

// Whole numbers ordered as the floats are; -0 equals 0, NaN above everything.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0xffffffffu;
  const uint32_t b = __float_as_uint(w == 0.0f ? 0.0f : w);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

struct SelectShared {
  uint32_t hist[kBins * kHistCopies];
  uint32_t place[kHeld * kSelectWaves];  // kept before each 64 slots, two counts in one word
  __align__(16) uint32_t wave_sum[kSelectWaves];
  uint32_t prefix, need;
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
__device__ __forceinline__ uint32_t scan_u32(uint32_t v, int lane) {
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    const uint32_t up = __shfl_up(v, o);
    if (lane >= o) v += up;
  }
  return v;
}

__global__ __launch_bounds__(kSelectThreads) void select_kernel(EvictArgs a) {
  __shared__ SelectShared sh;
  const int H = a.c.heads;
  const int s = blockIdx.x / H, h = blockIdx.x - s * H;
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  int64_t n64 = a.c.lens[s];
  const int64_t most = (int64_t)a.c.table_width * a.c.page.d;
  n64 = n64 < 0 ? 0 : (n64 > most ? most : n64);
  const int n = (int)n64;
  int32_t *kept = a.kept + ((int64_t)s * H + h) * a.budget;
  if (h == 0 && tid == 0) a.new_lens[s] = n < a.budget ? n : a.budget;
  if (n <= a.budget) {
    for (int r = tid; r < a.budget; r += kSelectThreads) kept[r] = r < n ? r : -1;
    return;
  }
  const int sink = a.sink, recent = a.recent, M = n - sink - recent, need0 = a.budget - sink - recent;
  for (int r = tid; r < sink; r += kSelectThreads) kept[r] = r;
  for (int r = tid; r < recent; r += kSelectThreads) kept[a.budget - recent + r] = n - recent + r;
  if (need0 == 0) return;
  const int32_t *trow = a.c.table + (int64_t)s * a.c.table_stride;
  const int segments = (M + kSegment - 1) / kSegment;
  // keys of slots segment + tid + 1024 u: an absent slot's is 0, the least
  uint32_t key[kHeld];
  const auto load = [&](int from) {
#pragma unroll
    for (int b = 0; b < kHeld; b += kBatch) {
      if (from + b * kSelectThreads >= M) break;
      SlotPlace p[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int i = from + (b + u) * kSelectThreads + tid;
        p[u] = SlotPlace{-1, 0};
        if (i < M) p[u] = slot_place(a.c, trow, (uint32_t)(sink + i));
      }
      float w[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        w[u] = 0.0f;
        if (p[u].page >= 0) w[u] = a.c.weights[((int64_t)p[u].page * H + h) * a.c.page.d + p[u].row];
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) key[b + u] = p[u].page < 0 ? 0u : weight_key(w[u]);
    }
  };

  // the need-th largest key, digit by digit
  uint32_t prefix = 0, need = (uint32_t)need0;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), bits = pass == 2 ? 10 : 11;
    for (int i = tid; i < kBins * kHistCopies / 4; i += kSelectThreads) ((u32x4 *)sh.hist)[i] = (u32x4){0, 0, 0, 0};
    __syncthreads();
#pragma unroll 1
    for (int from = 0; from < M; from += kSegment) {
      if (pass == 0 || segments > 1) load(from);
#pragma unroll
      for (int u = 0; u < kHeld; ++u) {
        const int at = from + u * kSelectThreads;
        if (at >= M) break;
        const bool in = at + tid < M && (pass == 0 || (key[u] >> (shift + bits)) == (prefix >> (shift + bits)));
        const uint32_t bin = (key[u] >> shift) & ((1u << bits) - 1u);
        const uint64_t who = __ballot(in);
        if (!who) continue;
        const uint32_t one = __builtin_amdgcn_readlane(bin, __ffsll((unsigned long long)who) - 1);
        if (__ballot(in && bin != one) == 0) {
          if (lane == 0) atomicAdd(&sh.hist[one * kHistCopies], (uint32_t)__popcll(who));
        } else if (in) {
          atomicAdd(&sh.hist[bin * kHistCopies + (lane & (kHistCopies - 1))], 1u);
        }
      }
    }
    __syncthreads();
    // thread t has the counts 2 t and 2 t + 1 from the top
    uint32_t cnt[2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const u32x4 *c = (const u32x4 *)&sh.hist[(kBins - 1 - (2 * tid + b)) * kHistCopies];
      const u32x4 x = c[0] + c[1];
      cnt[b] = (x[0] + x[1]) + (x[2] + x[3]);
    }
    const uint32_t own = cnt[0] + cnt[1], upto = scan_u32(own, lane);
    if (lane == kWave - 1) sh.wave_sum[wave] = upto;
    __syncthreads();
    uint32_t total;
    uint32_t above = upto - own + before_wave(sh.wave_sum, wave, &total);
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      if (above < need && need <= above + cnt[b]) {
        sh.prefix = prefix | ((uint32_t)(kBins - 1 - (2 * tid + b)) << shift);
        sh.need = need - above;
      }
      above += cnt[b];
    }
    __syncthreads();
    prefix = sh.prefix;
    need = sh.need;
  }
  // keys above `prefix` are kept, and the first `need` of those equal to it
  uint32_t base_gt = 0, base_eq = 0;
#pragma unroll 1
  for (int from = 0; from < M; from += kSegment) {
    if (segments > 1) load(from);
#pragma unroll
    for (int u = 0; u < kHeld; ++u) {
      const int at = from + u * kSelectThreads;
      const bool in = at + tid < M;
      const uint64_t gt = __ballot(in && key[u] > prefix), eq = __ballot(in && key[u] == prefix);
      if (lane == 0) sh.place[u * kSelectWaves + wave] = (uint32_t)__popcll(gt) | ((uint32_t)__popcll(eq) << 16);
    }
    __syncthreads();
    // 512 counts in slot order, each half at most 32,768 in all
    uint32_t own = 0, upto = 0, total;
    if (tid < kHeld * kSelectWaves) own = sh.place[tid];
    upto = scan_u32(own, lane);
    if (lane == kWave - 1) sh.wave_sum[wave] = upto;
    __syncthreads();
    upto += before_wave(sh.wave_sum, wave, &total);
    if (tid < kHeld * kSelectWaves) sh.place[tid] = upto - own;
    __syncthreads();
    const uint64_t below = ((uint64_t)1 << lane) - 1;
#pragma unroll
    for (int u = 0; u < kHeld; ++u) {
      const int at = from + u * kSelectThreads;
      if (at >= M) break;
      const bool in = at + tid < M, is_gt = in && key[u] > prefix, is_eq = in && key[u] == prefix;
      const uint32_t pre = sh.place[u * kSelectWaves + wave];
      const uint32_t gt = base_gt + (pre & 0xffffu) + __popcll(__ballot(is_gt) & below);
      const uint32_t eq = base_eq + (pre >> 16) + __popcll(__ballot(is_eq) & below);
      if (is_gt || (is_eq && eq < need)) kept[sink + gt + (eq < need ? eq : need)] = sink + at + tid;
    }
    base_gt += total & 0xffffu;
    base_eq += total >> 16;
    __syncthreads();
  }
}

// One thread per 16-byte piece of a kept slot's key row, and the same piece of its value row.
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
  const u32x4 k = *(const u32x4 *)(a.c.k + fo);
  const u32x4 v = *(const u32x4 *)(a.c.v + fo);
  *(u32x4 *)(a.c.k + dst) = k;
  *(u32x4 *)(a.c.v + dst) = v;
  if (piece == 0)
    a.c.weights[((int64_t)to.page * a.c.heads + h) * a.c.page.d + to.row] =
        a.c.weights[((int64_t)from.page * a.c.heads + h) * a.c.page.d + from.row];
}

}  // namespace

void launch_evict(const EvictArgs &a, hipStream_t st) {
  select_kernel<<<dim3((unsigned)(a.c.seqs * a.c.heads)), kSelectThreads, 0, st>>>(a);
  const int pieces = a.c.dim * a.itemsize / 16;
  const int64_t total = (int64_t)a.c.seqs * a.c.heads * a.budget * pieces;
  move_kernel<<<dim3((unsigned)((total + 255) / 256)), 256, 0, st>>>(a, pieces, total);
}

}  // namespace kmi
