// adjust_logits.hip -- logits by a text's penalties, biases and masks.
//
//   z = l;  seen: z > 0 ? z / r : z r;  z -= f c + (c > 0 ? p : 0);  z += bias;  masked: z = -inf
//
// A row sees its sequence's text up to its own token.  A work-group has a piece of a row's vocabulary: it counts the
// text's tokens of that piece in LDS (whole numbers, so the order of the additions does not matter), notes which bias of
// the list each entry takes (the largest place, so the last of equal ones), then goes over the logits once.  Few
// entries of a piece are touched; those are computed in 64 bits one after the other, the others pass by.
#include "step.h"

namespace kmi {
namespace {

constexpr uint32_t kInPrompt = 0x80000000u;
constexpr int kChunk = 8;                    // entries of a thread at a time

template <class T> struct Logit;
template <> struct Logit<Bf16> {
  typedef uint16_t E;
  static __device__ __forceinline__ float get(E x) { return __uint_as_float((uint32_t)x << 16); }
  static __device__ __forceinline__ E put(float x) { return (E)Bf16::pack(x, x); }
};
template <> struct Logit<F16> {
  typedef uint16_t E;
  static __device__ __forceinline__ float get(E x) { return (float)__builtin_bit_cast(_Float16, x); }
  static __device__ __forceinline__ E put(float x) { return (E)F16::pack(x, x); }
};
template <> struct Logit<float> {
  typedef float E;
  static __device__ __forceinline__ float get(E x) { return x; }
  static __device__ __forceinline__ E put(float x) { return x; }
};

template <class T>
__global__ __launch_bounds__(kLogitThreads) void adjust_kernel(LogitArgs a) {
  typedef typename Logit<T>::E E;
  constexpr int kWords = kChunk * sizeof(E) / 16;
  extern __shared__ uint32_t table[];        // [piece] counts with text, then [piece] places with biases
  const int tid = threadIdx.x;
  const int pieces = (a.vocab + a.piece - 1) / a.piece;
  const int64_t t = blockIdx.x / pieces;
  const int i0 = (int)(blockIdx.x - t * pieces) * a.piece, i1 = i0 + a.piece < a.vocab ? i0 + a.piece : a.vocab;
  const int s = owner_of(a.starts, a.seqs, t);
  int64_t begin = a.starts[s], end = a.starts[s + 1];
  begin = begin < 0 ? 0 : begin;
  end = end > a.rows ? a.rows : end;
  if (t < begin || t >= end) return;
  uint32_t *counts = table, *which = table + (a.text ? a.piece : 0);
  const int entries = a.piece * ((a.text ? 1 : 0) + (a.biases ? 1 : 0));
  for (int i = tid * 4; i < entries; i += kLogitThreads * 4) *(u32x4 *)(table + i) = (u32x4){0, 0, 0, 0};
  __syncthreads();
  double rep = 1.0, pres = 0.0, freq = 0.0;
  if (a.text) {
    if (a.repetition) rep = (double)a.repetition[s];
    if (a.presence) pres = (double)a.presence[s];
    if (a.frequency) freq = (double)a.frequency[s];
    int64_t n = a.lens[s] - (end - t) + 1;   // tokens up to the row's own
    n = n < a.text_width ? n : a.text_width;
    const int prompt = a.prompt_lens ? a.prompt_lens[s] : 0;
    const int32_t *text = a.text + s * a.text_stride;
    for (int64_t i = tid; i < n; i += kLogitThreads) {
      const int x = text[i];
      if (x < i0 || x >= i1) continue;
      if (i < prompt) atomicOr(&counts[x - i0], kInPrompt);
      else atomicAdd(&counts[x - i0], 1u);
    }
  }
  for (int i = tid; i < a.biases; i += kLogitThreads) {
    const int x = a.bias_tokens[(int64_t)s * a.biases + i];
    if (x >= i0 && x < i1) atomicMax(&which[x - i0], (uint32_t)i + 1u);
  }
  __syncthreads();
  const double inverse = 1.0 / rep;
  const E *in = (const E *)a.logits + t * a.stride;
  E *out = (E *)a.out + t * a.out_stride;
  const uint32_t *mask = a.mask ? a.mask + t * a.mask_stride : nullptr;
  for (int x0 = i0 + tid * kChunk; x0 < i1; x0 += kLogitThreads * kChunk) {
    const bool full = a.whole && x0 + kChunk <= i1;
    union { u32x4 w[kWords]; E e[kChunk]; } u;
    if (full) {
#pragma unroll
      for (int k = 0; k < kWords; ++k) u.w[k] = ((const u32x4 *)(in + x0))[k];
    } else {
#pragma unroll
      for (int k = 0; k < kChunk; ++k) u.e[k] = x0 + k < i1 ? in[x0 + k] : E(0);
    }
    uint32_t bits = 0xffu;
    if (mask) bits = (mask[x0 >> 5] >> (x0 & 31)) & 0xffu;
    uint32_t touched = 0;
#pragma unroll
    for (int k = 0; k < kChunk; ++k) {
      uint32_t any = 0;
      if (a.text) any |= counts[x0 - i0 + k];
      if (a.biases) any |= which[x0 - i0 + k];
      touched |= any ? 1u << k : 0u;
    }
    touched &= bits;
    while (touched) {
      const int k = __ffs(touched) - 1;
      touched &= touched - 1;
      float l = 0.0f;
#pragma unroll
      for (int m = 0; m < kChunk; ++m) l = m == k ? Logit<T>::get(u.e[m]) : l;
      double z = (double)l;
      const uint32_t c = a.text ? counts[x0 - i0 + k] : 0u;
      if (c) {
        if (z > 0.0) {
          double q = z * inverse;
          if (__builtin_fabs(q) < INFINITY) q = __builtin_fma(__builtin_fma(-q, rep, z), inverse, q);
          z = q;
        } else {
          z *= rep;
        }
        const uint32_t made = c & ~kInPrompt;
        if (made) z -= freq * (double)made + pres;
      }
      const uint32_t w = a.biases ? which[x0 - i0 + k] : 0u;
      if (w) z += (double)a.bias[(int64_t)s * a.biases + (w - 1)];
      const E e = Logit<T>::put((float)z);
#pragma unroll
      for (int m = 0; m < kChunk; ++m) u.e[m] = m == k ? e : u.e[m];
    }
    const E none = Logit<T>::put(-INFINITY);
#pragma unroll
    for (int k = 0; k < kChunk; ++k) u.e[k] = (bits >> k) & 1u ? u.e[k] : none;
    if (full) {
#pragma unroll
      for (int k = 0; k < kWords; ++k) ((u32x4 *)(out + x0))[k] = u.w[k];
    } else {
#pragma unroll
      for (int k = 0; k < kChunk; ++k)
        if (x0 + k < i1) out[x0 + k] = u.e[k];
    }
  }
}

}  // namespace

void launch_adjust_logits(const LogitArgs &a, int type, dim3 grid, hipStream_t st) {
  const size_t lds = (size_t)a.piece * 4 * ((a.text ? 1 : 0) + (a.biases ? 1 : 0));
  if (type == CT_BF16) adjust_kernel<Bf16><<<grid, kLogitThreads, lds, st>>>(a);
  else if (type == CT_F16) adjust_kernel<F16><<<grid, kLogitThreads, lds, st>>>(a);
  else adjust_kernel<float><<<grid, kLogitThreads, lds, st>>>(a);
}

}  // namespace kmi
