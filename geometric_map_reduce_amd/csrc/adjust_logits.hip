// adjust_logits.hip -- logits by a text's penalties, biases and masks.
//
//   z = l;  seen: z > 0 ? z / r : z r;  z -= f c + (c > 0 ? p : 0);  z += bias;  masked: z = -inf
//
// A row sees its sequence's text up to its own token.  A work-group has a piece of a row: with the logits on their way it
// counts the text's tokens of its piece in LDS (whole numbers, so the order of the additions does not matter) and
// marks the entries that the list of biases names, then goes over the logits once.  Few entries of a piece are touched;
// those are computed in 64 bits one after the other, the others pass by.
// 158 rows of 131,072 bf16 entries with texts of up to 4,096 tokens take 28 us, 16 without rules, where a copy takes 12
// to 18, by whether the cache still holds them: the text's way through LDS comes before the first store.  Pieces of 16,384
// took 35 us; rows that share a sequence's table, one after the other in a work-group, 33, and twice as long for
// those of the longest draft.
#include "step.h"

namespace kmi {
namespace {

// An entry's word: seen in the prompt, named by the list of biases, and how often it was seen past the prompt (a
// text has less than 2^30 tokens).
constexpr uint32_t kInPrompt = 0x80000000u, kBiased = 0x40000000u, kMade = 0x3fffffffu;
constexpr int kChunk = 8;                    // entries of a thread at a time
constexpr int kStrip = 512;                  // a wave's entries at a time
constexpr int kListed = 512;                 // biases of a piece that are held in LDS

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

// CHUNKS: of a row's piece for each thread.
template <class T, int CHUNKS>
__global__ __launch_bounds__(kLogitThreads, 8) void adjust_kernel(LogitArgs a) {
  typedef typename Logit<T>::E E;
  constexpr int kWords = kChunk * sizeof(E) / 16, kPiece = CHUNKS * kChunk * kLogitThreads;
  __shared__ __align__(16) uint32_t table[kPiece];
  __shared__ __align__(16) int listed_token[kListed];
  __shared__ int listed_at[kListed], listed;
  __shared__ float listed_bias[kListed];
  const int tid = threadIdx.x;
  const int pieces = (a.vocab + kPiece - 1) / kPiece;
  const int64_t t = blockIdx.x / pieces;
  const int piece = (int)(blockIdx.x - t * pieces), V = a.vocab;
  const int s = owner_of(a.starts, a.seqs, t);
  int64_t begin = a.starts[s], end = a.starts[s + 1];
  begin = begin < 0 ? 0 : begin;
  end = end > a.rows ? a.rows : end;
  if (t < begin || t >= end) return;         // of no sequence

  // Strips of 512 entries are dealt to the pieces in turn: a text's common tokens lie close together.
  const auto entry = [&](int c) {            // the first of the thread's chunk c, whose word is at c * 4096 + 8 tid
    const int strip = (c * kLogitThreads + tid) * kChunk / kStrip;
    return (int64_t)(strip * pieces + piece) * kStrip + tid * kChunk % kStrip;
  };
  const auto place = [&](int x) {            // where x's word is; -1: another piece's
    const int strip = x / kStrip, mine = (int)fast_div(a.pieces_div, (uint32_t)strip);
    return x >= 0 && x < V && strip - mine * pieces == piece ? mine * kStrip + x % kStrip : -1;
  };
  // the piece and its mask, on their way while the table is made
  union Held { u32x4 w[kWords]; E e[kChunk]; };
  Held u[CHUNKS];
  uint32_t bits[CHUNKS];
  const E *in = (const E *)a.logits + t * a.stride;
  const uint32_t *mask = a.mask ? a.mask + t * a.mask_stride : nullptr;
#pragma unroll
  for (int c = 0; c < CHUNKS; ++c) {
    const int64_t x0 = entry(c);
    if (a.whole && x0 + kChunk <= V) {
#pragma unroll
      for (int k = 0; k < kWords; ++k) u[c].w[k] = ((const u32x4 *)(in + x0))[k];
    } else {
#pragma unroll
      for (int k = 0; k < kChunk; ++k) u[c].e[k] = x0 + k < V ? in[x0 + k] : E(0);
    }
    bits[c] = mask && x0 < V ? mask[x0 >> 5] >> (x0 & 31) : 0xffu;
  }
  const bool rules = a.text || a.biases;
  double rep = 1.0, pres = 0.0, freq = 0.0;
  int prompt = 0;
  const int32_t *text = a.text + s * a.text_stride;
  const auto count = [&](int x, int64_t i) {
    const int at = place(x);
    if (at < 0) return;
    if (i < prompt) atomicOr(&table[at], kInPrompt);
    else atomicAdd(&table[at], 1u);
  };
  if (rules) {
    for (int i = tid * 4; i < kPiece; i += kLogitThreads * 4) *(u32x4 *)(table + i) = (u32x4){0, 0, 0, 0};
    if (tid == 0) listed = 0;
    for (int i = tid; i < kListed; i += kLogitThreads) listed_token[i] = -1;
    __syncthreads();
    if (a.text) {
      if (a.repetition) rep = (double)a.repetition[s];
      if (a.presence) pres = (double)a.presence[s];
      if (a.frequency) freq = (double)a.frequency[s];
      if (a.prompt_lens) prompt = a.prompt_lens[s];
      const int64_t n = a.lens[s] - (end - t) + 1;       // tokens up to the row's own
      const int64_t m = n < a.text_width ? n : a.text_width;
      if (((uintptr_t)text & 15) == 0) {
        for (int64_t i = 4 * tid; i < m; i += 4 * kLogitThreads) {
          if (i + 4 <= m) {
            const u32x4 four = *(const u32x4 *)(text + i);
#pragma unroll
            for (int k = 0; k < 4; ++k) count((int)four[k], i + k);
          } else {
            for (int k = 0; i + k < m; ++k) count(text[i + k], i + k);
          }
        }
      } else {
        for (int64_t i = tid; i < m; i += kLogitThreads) count(text[i], i);
      }
    }
    for (int i = tid; i < a.biases; i += kLogitThreads) {
      const int x = a.bias_tokens[(int64_t)s * a.biases + i], word = place(x);
      if (word < 0) continue;
      atomicOr(&table[word], kBiased);
      const int at = atomicAdd(&listed, 1);
      if (at < kListed) {
        listed_token[at] = x;
        listed_at[at] = i;
        listed_bias[at] = a.bias[(int64_t)s * a.biases + i];
      }
    }
    __syncthreads();
  }
  const double inverse = 1.0 / rep;
  // of equal biases the last in the list, whichever order they came to LDS in
  const int biases = listed;
  const auto bias_of = [&](int x) {
    int last = -1;
    float v = 0.0f;
    if (biases <= kListed) {
      for (int i = 0; i < biases; i += 4) {
        const u32x4 four = *(const u32x4 *)(listed_token + i);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if ((int)four[k] == x && listed_at[i + k] > last) {
            last = listed_at[i + k];
            v = listed_bias[i + k];
          }
      }
    } else {
      for (int i = a.biases - 1; i >= 0 && last < 0; --i)
        if (a.bias_tokens[(int64_t)s * a.biases + i] == x) last = i;
      v = a.bias[(int64_t)s * a.biases + last];
    }
    return (double)v;
  };
  const E none = Logit<T>::put(-INFINITY);
  E *out = (E *)a.out + t * a.out_stride;
#pragma unroll
  for (int c = 0; c < CHUNKS; ++c) {
    const int64_t x0 = entry(c);
    const int word = (c * kLogitThreads + tid) * kChunk;
    if (x0 >= V) break;
    uint32_t touched = 0;
    if (rules) {
      const u32x4 lo = *(const u32x4 *)(table + word), hi = *(const u32x4 *)(table + word + 4);
#pragma unroll
      for (int k = 0; k < 4; ++k) touched |= (lo[k] ? 1u << k : 0u) | (hi[k] ? 16u << k : 0u);
      touched &= bits[c];
    }
    while (touched) {
      const int k = __ffs(touched) - 1;
      touched &= touched - 1;
      float l = 0.0f;
#pragma unroll
      for (int m = 0; m < kChunk; ++m) l = m == k ? Logit<T>::get(u[c].e[m]) : l;
      double z = (double)l;
      const uint32_t w = table[word + k];
      if (w & (kInPrompt | kMade)) {
        if (z > 0.0) {
          double q = z * inverse;            // an exact quotient comes out exact
          if (__builtin_fabs(q) < INFINITY && q != 0.0) q = __builtin_fma(__builtin_fma(-q, rep, z), inverse, q);
          z = q;
        } else {
          z *= rep;
        }
        if (w & kMade) z -= freq * (double)(w & kMade) + pres;
      }
      if (w & kBiased) z += bias_of((int)x0 + k);
      const E e = Logit<T>::put((float)z);
#pragma unroll
      for (int m = 0; m < kChunk; ++m) u[c].e[m] = m == k ? e : u[c].e[m];
    }
#pragma unroll
    for (int k = 0; k < kChunk; ++k) u[c].e[k] = (bits[c] >> k) & 1u ? u[c].e[k] : none;
    if (a.whole && x0 + kChunk <= V) {
#pragma unroll
      for (int k = 0; k < kWords; ++k) ((u32x4 *)(out + x0))[k] = u[c].w[k];
    } else {
#pragma unroll
      for (int k = 0; k < kChunk; ++k)
        if (x0 + k < V) out[x0 + k] = u[c].e[k];
    }
  }
}

template <class T>
void launch_type(const LogitArgs &a, dim3 grid, hipStream_t st) {
  if (a.piece == kLogitPiece) adjust_kernel<T, 2><<<grid, kLogitThreads, 0, st>>>(a);
  else adjust_kernel<T, 1><<<grid, kLogitThreads, 0, st>>>(a);
}

}  // namespace

void launch_adjust_logits(const LogitArgs &a, int type, dim3 grid, hipStream_t st) {
  if (type == CT_BF16) launch_type<Bf16>(a, grid, st);
  else if (type == CT_F16) launch_type<F16>(a, grid, st);
  else launch_type<float>(a, grid, st);
}

}  // namespace kmi
