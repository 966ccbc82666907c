// paged_evict.hip -- eviction from a paged cache by attention weight.
//
// Of a sequence's n slots each key/value head keeps `budget`: the first `sink`, the last
// `recent`, and of those between the ones with the largest weights (equal weights: the lower
// slot).  Kept slots move, in their order, to slots 0 .. of the pages in new_table, keys,
// values and weights alike; n <= budget keeps them all.
//
// Selection: one work-group per (sequence, head) finds the smallest kept weight by three passes
// over 11, 11 and 10 bits of an order-preserving whole number (counts in LDS; integers, so the
// order of the additions does not matter), then one scan of counts gives every slot its place.
// It is bound by the latency of its steps: page numbers and weights are loaded eight at a time,
// and a wave whose lanes all meet one count adds to it once (cleared weights are all equal).
// The move is a second kernel, one 16-byte piece of a key and of a value row per thread, bound
// by HBM.
#include "paged.h"

namespace kmi {
namespace {

constexpr int kSelectThreads = 1024;
constexpr int kSelectWaves = kSelectThreads / kWave;
constexpr int kBins = 2048;             // counts of a pass
constexpr int kHistCopies = 2;          // even and odd lanes: fewer collisions
constexpr int kSelectCache = 32768;     // weights held in LDS (132 KB); longer rows are read again
constexpr int kBatch = 8;

// Whole numbers ordered as the floats are; -0 equals 0, NaN above everything.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0xffffffffu;
  const uint32_t b = __float_as_uint(w == 0.0f ? 0.0f : w);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

struct SelectShared {
  uint32_t hist[kBins * kHistCopies];
  uint32_t wave_gt[kSelectWaves], wave_eq[kSelectWaves];
  uint32_t prefix, need;
};

// One spare word after every 32 keeps threads that read at a stride of a power of two apart.
__device__ __forceinline__ int cache_at(int i) { return i + (i >> 5); }

__global__ __launch_bounds__(kSelectThreads) void select_kernel(EvictArgs a, int cache_words) {
  __shared__ SelectShared sh;
  extern __shared__ uint32_t cache[];
  const int H = a.c.heads;
  const int s = blockIdx.x / H, h = blockIdx.x - s * H;
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
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
  // eight keys, slots first + 1024 u: an absent slot's is 0, the least
  const auto load = [&](int first, uint32_t *k) {
    SlotPlace p[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int i = first + u * kSelectThreads;
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
    for (int u = 0; u < kBatch; ++u) k[u] = p[u].page < 0 ? 0u : weight_key(w[u]);
  };
  const bool held = cache_at(M - 1) < cache_words;
  if (held) {
    for (int i = tid; i < M; i += kBatch * kSelectThreads) {
      uint32_t k[kBatch];
      load(i, k);
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        if (i + u * kSelectThreads < M) cache[cache_at(i + u * kSelectThreads)] = k[u];
    }
  }
  const auto key = [&](int i) -> uint32_t {
    if (held) return cache[cache_at(i)];
    const SlotPlace p = slot_place(a.c, trow, (uint32_t)(sink + i));
    return p.page < 0 ? 0u : weight_key(a.c.weights[((int64_t)p.page * H + h) * a.c.page.d + p.row]);
  };

  // the need-th largest key, digit by digit
  uint32_t prefix = 0, need = (uint32_t)need0;
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), bits = pass == 2 ? 10 : 11;
    for (int i = tid; i < kBins * kHistCopies; i += kSelectThreads) sh.hist[i] = 0;
    __syncthreads();
    for (int base = tid; base - tid < M; base += kBatch * kSelectThreads) {
      uint32_t k[kBatch];
      if (held) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          const int i = base + u * kSelectThreads;
          k[u] = i < M ? cache[cache_at(i)] : 0u;
        }
      } else {
        load(base, k);
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const bool in = base + u * kSelectThreads < M && (pass == 0 || (k[u] >> (shift + bits)) == (prefix >> (shift + bits)));
        const uint32_t bin = (k[u] >> shift) & ((1u << bits) - 1u);
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
      const int bin = kBins - 1 - (2 * tid + b);
      cnt[b] = sh.hist[bin * kHistCopies] + sh.hist[bin * kHistCopies + 1];
    }
    const uint32_t own = cnt[0] + cnt[1];
    uint32_t upto = own;
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
      const uint32_t up = __shfl_up(upto, o);
      if (lane >= o) upto += up;
    }
    if (lane == kWave - 1) sh.wave_gt[wave] = upto;
    __syncthreads();
    for (int w = 0; w < wave; ++w) upto += sh.wave_gt[w];
    uint32_t above = upto - own;
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
  // keys above `prefix` are kept, and the first `need` of those equal to it.  Each thread owns
  // a run of slots; one scan of both counts gives its places.
  const int L = (M + kSelectThreads - 1) / kSelectThreads;
  const int i0 = tid * L < M ? tid * L : M, i1 = i0 + L < M ? i0 + L : M;
  uint32_t gt = 0, eq = 0;
  for (int i = i0; i < i1; ++i) {
    const uint32_t k = key(i);
    gt += k > prefix;
    eq += k == prefix;
  }
  uint32_t sgt = gt, seq = eq;
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    const uint32_t ug = __shfl_up(sgt, o), ue = __shfl_up(seq, o);
    if (lane >= o) { sgt += ug; seq += ue; }
  }
  if (lane == kWave - 1) { sh.wave_gt[wave] = sgt; sh.wave_eq[wave] = seq; }
  __syncthreads();
  for (int w = 0; w < wave; ++w) { sgt += sh.wave_gt[w]; seq += sh.wave_eq[w]; }
  uint32_t bgt = sgt - gt, beq = seq - eq;
  for (int i = i0; i < i1; ++i) {
    const uint32_t k = key(i);
    if (k > prefix || (k == prefix && beq < need)) kept[sink + bgt + (beq < need ? beq : need)] = sink + i;
    bgt += k > prefix;
    beq += k == prefix;
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

int launch_evict(const EvictArgs &a, hipStream_t st) {
  const int64_t most = (int64_t)a.c.table_width * a.c.page.d;
  const int64_t keys = most < kSelectCache ? most : kSelectCache;
  const int words = (int)(keys + keys / 32 + 1);
  const size_t bytes = (size_t)words * sizeof(uint32_t);
  if (bytes > 32768 &&
      hipFuncSetAttribute((const void *)select_kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) != hipSuccess)
    return -1;
  select_kernel<<<dim3((unsigned)(a.c.seqs * a.c.heads)), kSelectThreads, bytes, st>>>(a, words);
  const int pieces = a.c.dim * a.itemsize / 16;
  const int64_t total = (int64_t)a.c.seqs * a.c.heads * a.budget * pieces;
  move_kernel<<<dim3((unsigned)((total + 255) / 256)), 256, 0, st>>>(a, pieces, total);
  return 0;
}

}  // namespace kmi
