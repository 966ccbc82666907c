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
// distance between neighbouring borders.  One read of two rows of the vocabulary: latency and
// one compute unit's read rate bound it.
#include "paged.h"

namespace kmi {
namespace {

constexpr int kVerifyThreads = 1024;
constexpr int kVerifyWaves = kVerifyThreads / kWave;

__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) v += __shfl_xor(v, o);
  return v;
}

// Mass of index i: what the next token is drawn from.
struct Mass {
  const float *p, *q;    // q null: the whole of p, but for index `skip`
  int skip;
  __device__ __forceinline__ double operator()(int i) const {
    double m = (double)p[i];
    if (q) m -= (double)q[i];
    if (i == skip) m = 0.0;
    return m > 0.0 ? m : 0.0;
  }
};

__global__ __launch_bounds__(kVerifyThreads) void verify_kernel(VerifyArgs a) {
  __shared__ double wave_total[kVerifyWaves];
  const int s = blockIdx.x, lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int K = a.drafts, V = a.vocab;
  int n = a.counts[s];
  n = n < 0 ? 0 : (n > K ? K : n);
  // every wave finds the first refusal by itself, 64 drafted tokens at a time
  int r = n;
  for (int base = 0; base < n; base += kWave) {
    const int i = base + lane;
    bool refused = false;
    if (i < n) {
      const int x = a.tokens[(int64_t)s * K + i];
      double px = 0.0, qx = 1.0;
      if (x >= 0 && x < V) {
        px = (double)a.target[((int64_t)s * (K + 1) + i) * V + x];
        if (a.draft) qx = (double)a.draft[((int64_t)s * K + i) * V + x];
      }
      refused = !((double)a.u_accept[(int64_t)s * K + i] * qx < px);
    }
    const uint64_t who = __ballot(refused);
    if (who) {
      r = base + __ffsll((unsigned long long)who) - 1;
      break;
    }
  }
  Mass mass{a.target + ((int64_t)s * (K + 1) + r) * V, nullptr, -1};
  if (r < n) {
    if (a.draft) mass.q = a.draft + ((int64_t)s * K + r) * V;
    else mass.skip = a.tokens[(int64_t)s * K + r];
  }
  // wave w owns indices [w L, (w + 1) L)
  const int L = ((V + kVerifyWaves - 1) / kVerifyWaves + kWave - 1) / kWave * kWave;
  const int i0 = wave * L < V ? wave * L : V, i1 = i0 + L < V ? i0 + L : V;
  int owner = -1;           // the wave whose range holds the goal
  double goal = 0.0, before = 0.0;
  for (int attempt = 0; attempt < 2; ++attempt) {
    double sum = 0.0;
    for (int i = i0 + lane; i < i1; i += kWave) sum += mass(i);
    sum = wave_sum_f64(sum);
    __syncthreads();
    if (lane == 0) wave_total[wave] = sum;
    __syncthreads();
    double total = 0.0;
    for (int w = 0; w < kVerifyWaves; ++w) total += wave_total[w];
    goal = (double)a.u_sample[s] * total;
    if (total > 0.0 || (!mass.q && mass.skip < 0)) break;
    mass.q = nullptr;       // nothing left over: the target's own row
    mass.skip = -1;
  }
  double run = 0.0;
  int last = -1;
  for (int w = 0; w < kVerifyWaves; ++w) {
    if (wave_total[w] > 0.0) last = w;
    if (owner < 0 && run + wave_total[w] > goal) {
      owner = w;
      before = run;
    }
    run += wave_total[w];
  }
  if (owner < 0) {          // u of 1 or more: the last index with mass
    owner = last;
    goal = 1.0 / 0.0;
  }
  if (wave == (owner < 0 ? 0 : owner)) {
    // the last index with mass stands in where rounding leaves every running sum at or below the goal
    int pick = V - 1;
    double c = before;
    for (int i = i0; i < i1 && owner >= 0; i += kWave) {
      const double m = i + lane < i1 ? mass(i + lane) : 0.0;
      double up = m;
#pragma unroll
      for (int o = 1; o < kWave; o <<= 1) {
        const double u = __shfl_up(up, o);
        if (lane >= o) up += u;
      }
      up += c;
      const uint64_t has = __ballot(m > 0.0), over = __ballot(m > 0.0 && up > goal);
      if (over) {
        pick = i + __ffsll((unsigned long long)over) - 1;
        break;
      }
      if (has) pick = i + 63 - __clzll((long long)has);
      c = __shfl(up, kWave - 1);
    }
    if (lane == 0) {
      a.out[(int64_t)s * (K + 1) + r] = pick;
      a.accepted[s] = r;
    }
  }
  for (int i = threadIdx.x; i <= K; i += kVerifyThreads)
    if (i != r) a.out[(int64_t)s * (K + 1) + i] = i < r ? a.tokens[(int64_t)s * K + i] : -1;
}

}  // namespace

void launch_verify(const VerifyArgs &a, hipStream_t st) {
  verify_kernel<<<dim3((unsigned)a.seqs), kVerifyThreads, 0, st>>>(a);
}

}  // namespace kmi
