// verify_draft.hip -- drafted tokens against the target's probabilities.
//
// Sequence s proposes tokens x_0 .. x_{n-1}, drawn from q_r = draft[s, r], which the target
// model rates p_r = target[s, r].  Token r is taken while u_accept[s, r] q_r(x_r) < p_r(x_r);
// with r the first one that is not, the next token is drawn by inversion of the running sum of
//   max(p_r - q_r, 0)       after a refusal (p_r itself where that is zero everywhere)
//   p_n                     where all n were taken
// with u_sample[s]: the lowest index whose running sum exceeds u times the total.  A missing
// draft stands for certainty: q_r is 1 at x_r and 0 elsewhere.
//
// Running sums are in 64 bits: a 32-bit sum of 10^5 probabilities is off by more than the
// distance between neighbouring borders.
//
// Two kernels: sums of pieces of the row by many work-groups (one read of two rows of the
// vocabulary, bound by HBM for a batch and by latency for one sequence), then one work-group per
// sequence that finds the piece and looks through it.  64 sequences of 131,072 tokens: 11 us
// (67 MB at 6 TB/s, part of it from the cache) and 5 us; one of 32,000: 3.6 and 4.4 us.  One work-group
// per sequence for both took 146 us: a compute unit reads some 10 bytes a nanosecond here.
#include "paged.h"

namespace kmi {
namespace {

constexpr int kVerifyWaves = kVerifyThreads / kWave;
constexpr int kPer = kVerifyPiece / kVerifyThreads;     // indices of a thread in a piece's step

// The first refused of the n drafted tokens (n: none), found by every wave for itself.
__device__ __forceinline__ int first_refused(const VerifyArgs &a, int s, int n) {
  const int lane = threadIdx.x & (kWave - 1), K = a.drafts, V = a.vocab;
  for (int base = 0; base < n; base += kWave) {
    const int i = base + lane;
    bool refused = false;
    if (i < n) {
      const int x = a.tokens[(int64_t)s * K + i];
      refused = true;
      if (x >= 0 && x < V) {
        const double px = (double)a.target[((int64_t)s * (K + 1) + i) * V + x];
        const double qx = a.draft ? (double)a.draft[((int64_t)s * K + i) * V + x] : 1.0;
        refused = !((double)a.u_accept[(int64_t)s * K + i] * qx < px);
      }
    }
    const uint64_t who = __ballot(refused);
    if (who) return base + __ffsll((unsigned long long)who) - 1;
  }
  return n;
}

__device__ __forceinline__ int drafted(const VerifyArgs &a, int s) {
  const int n = a.counts[s];
  return n < 0 ? 0 : (n > a.drafts ? a.drafts : n);
}

// What the next token is drawn from: the target's row, less the draft's after a refusal.
struct Rows {
  const float *p, *q;    // q null: nothing to take off but at index `skip`
  int skip;
};
__device__ __forceinline__ Rows rows_of(const VerifyArgs &a, int s, int r, int n) {
  Rows x{a.target + ((int64_t)s * (a.drafts + 1) + r) * a.vocab, nullptr, -1};
  if (r < n) {
    if (a.draft) x.q = a.draft + ((int64_t)s * a.drafts + r) * a.vocab;
    else x.skip = a.tokens[(int64_t)s * a.drafts + r];
  }
  return x;
}
__device__ __forceinline__ double positive(double v) { return v > 0.0 ? v : 0.0; }

// Sums of piece b of sequence s: of what is left, and of the whole of the target's row.
__global__ __launch_bounds__(kVerifyThreads) void verify_sums_kernel(VerifyArgs a) {
  __shared__ double red[2][kVerifyWaves];
  const int s = blockIdx.x / a.pieces, b = blockIdx.x - s * a.pieces;
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  const int n = drafted(a, s), r = first_refused(a, s, n);
  const Rows x = rows_of(a, s, r, n);
  const int i0 = b * a.piece, i1 = i0 + a.piece < a.vocab ? i0 + a.piece : a.vocab;
  double left = 0.0, whole = 0.0;
  for (int i = i0 + tid; i < i1; i += kVerifyPiece) {
    float p[kPer], q[kPer];
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int k = i + u * kVerifyThreads;
      p[u] = k < i1 ? x.p[k] : 0.0f;
      q[u] = x.q && k < i1 ? x.q[k] : 0.0f;
      if (k == x.skip) q[u] = p[u];
    }
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      left += positive((double)p[u] - (double)q[u]);
      whole += positive((double)p[u]);
    }
  }
  left = wave_scan_f64(left);
  whole = wave_scan_f64(whole);
  if (lane == kWave - 1) {
    red[0][wave] = left;
    red[1][wave] = whole;
  }
  __syncthreads();
  if (tid == 0) {
    double l = 0.0, w = 0.0;
    for (int k = 0; k < kVerifyWaves; ++k) {
      l += red[0][k];
      w += red[1][k];
    }
    a.sums[(int64_t)s * a.pieces + b] = make_double2(l, w);
    if (b == 0) a.accepted[s] = r;
  }
}

__global__ __launch_bounds__(kVerifyThreads) void verify_pick_kernel(VerifyArgs a) {
  __shared__ double wave_total[kVerifyWaves];
  __shared__ int first, last;
  const int s = blockIdx.x, tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  const int K = a.drafts, V = a.vocab, r = a.accepted[s], n = drafted(a, s);
  if (tid == 0) {
    first = V;
    last = -1;
  }
  // every wave finds the piece that holds the goal: the first whose running sum passes it, or
  // the last with mass (u of 1 or more)
  double2 own = make_double2(0.0, 0.0);
  if (lane < a.pieces) own = a.sums[(int64_t)s * a.pieces + lane];
  const bool any = __any(own.x > 0.0);      // nothing left over: the target's own row
  const double mass = any ? own.x : own.y, upto = wave_scan_f64(mass);
  double goal = (double)a.u_sample[s] * __shfl(upto, kWave - 1);
  const uint64_t over = __ballot(mass > 0.0 && upto > goal), has = __ballot(mass > 0.0);
  int pick = V - 1;
  if (has) {                                 // the same in every wave
    const int b = over ? __ffsll((unsigned long long)over) - 1 : 63 - __clzll((long long)has);
    if (!over) goal = INFINITY;
    double before = b > 0 ? __shfl(upto, b - 1) : 0.0;
    Rows x = rows_of(a, s, r, n);
    if (!any) x = Rows{x.p, nullptr, -1};
    const int i0 = b * a.piece, i1 = i0 + a.piece < V ? i0 + a.piece : V;
    for (int base = i0; base < i1; base += kVerifyPiece) {
      // a thread's kPer indices in a row
      double m[kPer], sum = 0.0;
      const int i = base + tid * kPer;
#pragma unroll
      for (int u = 0; u < kPer; ++u) {
        const int k = i + u;
        const float p = k < i1 ? x.p[k] : 0.0f;
        float q = x.q && k < i1 ? x.q[k] : 0.0f;
        if (k == x.skip) q = p;
        m[u] = positive((double)p - (double)q);
        sum += m[u];
      }
      const double scan = wave_scan_f64(sum);
      __syncthreads();
      if (lane == kWave - 1) wave_total[wave] = scan;
      __syncthreads();
      double c = before + (scan - sum);
      for (int w = 0; w < wave; ++w) c += wave_total[w];
      for (int w = 0; w < kVerifyWaves; ++w) before += wave_total[w];
      int over_at = V, mass_at = -1;         // this thread's first index past the goal, last with mass
#pragma unroll
      for (int u = 0; u < kPer; ++u) {
        c += m[u];
        if (m[u] > 0.0) {
          if (c > goal && over_at == V) over_at = i + u;
          mass_at = i + u;
        }
      }
      // the lowest lane that has one, the highest that has one: one addition a wave
      const uint64_t past = __ballot(over_at < V), some = __ballot(mass_at >= 0);
      if (past && lane == __ffsll((unsigned long long)past) - 1) atomicMin(&first, over_at);
      if (some && lane == 63 - __clzll((long long)some)) atomicMax(&last, mass_at);
      __syncthreads();
      if (first < V) break;
    }
    // the last index with mass stands in where rounding leaves every running sum at or below the goal
    pick = first < V ? first : last;
  }
  for (int i = tid; i <= K; i += kVerifyThreads)
    a.out[(int64_t)s * (K + 1) + i] = i < r ? a.tokens[(int64_t)s * K + i] : (i == r ? pick : -1);
}

}  // namespace

void launch_verify(const VerifyArgs &a, hipStream_t st) {
  verify_sums_kernel<<<dim3((unsigned)(a.seqs * a.pieces)), kVerifyThreads, 0, st>>>(a);
  verify_pick_kernel<<<dim3((unsigned)a.seqs), kVerifyThreads, 0, st>>>(a);
}

}  // namespace kmi
