// rotary.hip -- rotary positions of token rows.
//
//   a' = factor (a cos t - b sin t),  b' = factor (a sin t + b cos t),  t = +-position freqs[i]
//
// for the pairs (a, b) of each head's first 2 pairs columns: columns i and i + pairs, or 2 i and 2 i + 1.
// The other columns are copied, or left where they are.  Every element is read once and written once.  An element is
// its own column times the cosine, added in one rounding to the other column's product, as it is where keys and
// queries turn on their way into a cache (paged_append_rotary.hip): the two give the same bits.
//
// A work-group has one or a few tokens.  Its threads first compute the tokens' cosines and sines, one each,
// into LDS (all heads share them), then go over the rows: a thread takes V pairs of a head at a time, two pieces
// of V columns, which makes it safe to write where it read.  Bound by HBM where there are many tokens: 16,384 tokens of
// 40 heads of 128 columns, 168 MB in and as many out, take 72.7 us (4.6 TB/s; a large copy reaches 4.8).
// 16 tokens of them are one launch's latency: 2.8 us on the GPU.
#include "step.h"

namespace kmi {
namespace {

template <class E, int V>
struct Piece {
  typedef E type __attribute__((ext_vector_type(V)));
};
template <class E>
struct Piece<E, 1> {
  typedef E type;
};

__device__ __forceinline__ float widen(uint16_t x, Bf16 *) { return __uint_as_float((uint32_t)x << 16); }
__device__ __forceinline__ float widen(uint16_t x, F16 *) { return (float)__builtin_bit_cast(_Float16, x); }
__device__ __forceinline__ float widen(float x, float *) { return x; }
__device__ __forceinline__ uint16_t narrow(float x, Bf16 *) { return (uint16_t)Bf16::pack(x, x); }
__device__ __forceinline__ uint16_t narrow(float x, F16 *) { return (uint16_t)F16::pack(held(x), 0.0f); }
__device__ __forceinline__ float narrow(float x, float *) { return x; }

// T: Bf16, F16 or float.  V: columns of a piece, a power of two that divides pairs and the columns left
// as they are, and whose pieces are aligned.
template <class T, class E, int V>
__global__ __launch_bounds__(kRotaryThreads) void rotary_kernel(RotaryArgs a) {
  typedef typename Piece<E, V>::type P;
  extern __shared__ float2 turned[];             // [tokens of the work-group][pairs]
  const int n = a.r.pairs;
  const int64_t t0 = (int64_t)blockIdx.x * a.tokens_wg;
  const int tokens = a.tokens - t0 < a.tokens_wg ? (int)(a.tokens - t0) : a.tokens_wg;
  for (int i = threadIdx.x; i < tokens * n; i += kRotaryThreads) {
    const int t = (int)fast_div(a.pairs_div, (uint32_t)i);
    const double2 cs = rotation(a.r, a.positions[t0 + t], i - t * n);
    turned[i] = make_float2((float)cs.x, (float)cs.y);
  }
  __syncthreads();
  // a head's pieces: n / V that turn, then the others
  const int items = tokens * a.heads * a.pieces;
  const int step = gridDim.y * kRotaryThreads;
  for (int id = blockIdx.y * kRotaryThreads + threadIdx.x; id < items; id += step) {
    const int row = (int)fast_div(a.pieces_div, (uint32_t)id), p = id - row * a.pieces;
    const int t = (int)fast_div(a.heads_div, (uint32_t)row), h = row - t * a.heads;
    const E *x = (const E *)a.x + (t0 + t) * a.x_stride + (int64_t)h * a.dim;
    E *y = (E *)a.out + (t0 + t) * a.out_stride + (int64_t)h * a.dim;
    if (p >= n / V) {
      const int at = 2 * n + (p - n / V) * V;
      *(P *)(y + at) = *(const P *)(x + at);
      continue;
    }
    const int ca = a.r.interleaved ? 2 * p * V : p * V, cb = a.r.interleaved ? ca + V : ca + n;
    union { P v; E e[V]; } u, w;
    u.v = *(const P *)(x + ca);
    w.v = *(const P *)(x + cb);
    const float2 *cs = turned + t * n + p * V;
    if (a.r.interleaved) {
      if constexpr (V == 1) {
        const float xa = widen(u.e[0], (T *)nullptr), xb = widen(w.e[0], (T *)nullptr);
        u.e[0] = narrow(fmaf(xa, cs[0].x, xb * -cs[0].y), (T *)nullptr);
        w.e[0] = narrow(fmaf(xb, cs[0].x, xa * cs[0].y), (T *)nullptr);
      } else {
#pragma unroll
        for (int k = 0; k < V; ++k) {
          // pair k lies in the first piece, or in the second
          E *e = k < V / 2 ? u.e + 2 * k : w.e + 2 * k - V;
          const float xa = widen(e[0], (T *)nullptr), xb = widen(e[1], (T *)nullptr);
          e[0] = narrow(fmaf(xa, cs[k].x, xb * -cs[k].y), (T *)nullptr);
          e[1] = narrow(fmaf(xb, cs[k].x, xa * cs[k].y), (T *)nullptr);
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const float xa = widen(u.e[k], (T *)nullptr), xb = widen(w.e[k], (T *)nullptr);
        u.e[k] = narrow(fmaf(xa, cs[k].x, xb * -cs[k].y), (T *)nullptr);
        w.e[k] = narrow(fmaf(xb, cs[k].x, xa * cs[k].y), (T *)nullptr);
      }
    }
    *(P *)(y + ca) = u.v;
    *(P *)(y + cb) = w.v;
  }
}

template <class T, class E>
void launch_type(const RotaryArgs &a, int v, dim3 grid, size_t lds, hipStream_t st) {
  if (v == 8) rotary_kernel<T, E, 8><<<grid, kRotaryThreads, lds, st>>>(a);
  else if (v == 4) rotary_kernel<T, E, 4><<<grid, kRotaryThreads, lds, st>>>(a);
  else if (v == 2) rotary_kernel<T, E, 2><<<grid, kRotaryThreads, lds, st>>>(a);
  else rotary_kernel<T, E, 1><<<grid, kRotaryThreads, lds, st>>>(a);
}

}  // namespace

void launch_rotary(const RotaryArgs &a, int type, int piece, dim3 grid, hipStream_t st) {
  const size_t lds = (size_t)a.tokens_wg * a.r.pairs * sizeof(float2);
  if (type == CT_BF16) launch_type<Bf16, uint16_t>(a, piece, grid, lds, st);
  else if (type == CT_F16) launch_type<F16, uint16_t>(a, piece, grid, lds, st);
  else launch_type<float, float>(a, piece, grid, lds, st);
}

}  // namespace kmi
