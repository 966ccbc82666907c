// adjust_logits.hip -- logits by a text's penalties, biases and masks.
//
//   z = l;  seen: z > 0 ? z / r : z r;  z -= f c + (c > 0 ? p : 0);  z += bias;  masked: z = -inf
//
// A row sees its sequence's text up to its own token.  A work-group has a piece of a row: with the logits, the mask, the
// text's first tokens and the biases on their way it clears a table in LDS, counts the text's tokens of its piece there
// (whole numbers, so the order of the additions does not matter), marks those and the entries that the list of biases
// names as bits, and goes over the logits once.  Few entries of a piece are touched; those are computed in 64 bits one
// after the other, the others pass by.
// 157 rows of 131,072 bf16 entries with texts of up to 4,096 tokens take 25 us, 14 without rules, where a copy takes 12
// to 18, by whether the cache still holds them: the text's way through LDS comes before the first store, 2,512
// work-groups of it, four to a compute unit.  Loads that had a condition of their own were each waited for, 28 us.  Pieces
// of 16,384 took 35 us; rows that share a sequence's table, one after the other in a work-group, 33, and twice as long for
// those of the longest draft; the touched entries in a list, one to a thread, with their logits read and written again
// 28, by way of the table 32.
#include "step.h"

namespace kmi {
namespace {

// An entry's word: seen in the prompt, named by the list of biases, and how often it was seen past the prompt (a
// text has less than 2^30 tokens).
constexpr uint32_t kInPrompt = 0x80000000u, kBiased = 0x40000000u, kMade = 0x3fffffffu;
constexpr int kChunk = 8;                    // entries of a thread at a time
constexpr int kStrip = 512;                  // a wave's entries at a time
// Lists of up to so many biases have those of the piece in LDS, to be looked through for each entry that one names: one
// row of 32,000 entries takes 5 us with 16 biases, 11 with 256.  Longer ones have for each entry of the piece its last place
// in the list, in as much LDS as the counts take: 6 us with 300, 10 with 10,000, where looking through the list took 5.9 ms.
constexpr int kListed = 256;

template <class T> struct Logit;
// put: rounded once, from 64 bits.
template <> struct Logit<Bf16> {
  typedef uint16_t E;
  static __device__ __forceinline__ float get(E x) { return __uint_as_float((uint32_t)x << 16); }
  static __device__ __forceinline__ E put(double x) {
    const float f = round_to_odd(x);
    return (E)Bf16::pack(f, f);
  }
};
template <> struct Logit<F16> {
  typedef uint16_t E;
  static __device__ __forceinline__ float get(E x) { return (float)__builtin_bit_cast(_Float16, x); }
  static __device__ __forceinline__ E put(double x) {
    const float f = round_to_odd(x);
    return (E)F16::pack(f, f);
  }
};
template <> struct Logit<float> {
  typedef float E;
  static __device__ __forceinline__ float get(E x) { return x; }
  static __device__ __forceinline__ E put(double x) { return (float)x; }
};

// A thread's entries.  Entry k, in a register that is not known beforehand, by selection.
template <class E>
union Held {
  static constexpr int kEach = 4 / sizeof(E), kRegs = kChunk / kEach;
  u32x4 w[kRegs / 4];
  uint32_t r[kRegs];
  E e[kChunk];
  __device__ __forceinline__ E at(int k) const {
    uint32_t x[kRegs];
#pragma unroll
    for (int i = 0; i < kRegs; ++i) x[i] = r[i];
    const int which = k / kEach;
#pragma unroll
    for (int n = kRegs / 2; n; n /= 2)
#pragma unroll
      for (int i = 0; i < n; ++i) x[i] = which & n ? x[i + n] : x[i];
    if constexpr (kEach == 2) return (E)(x[0] >> (k & 1) * 16);
    else return __uint_as_float(x[0]);
  }
  __device__ __forceinline__ void put(int k, E v) {
#pragma unroll
    for (int i = 0; i < kRegs; ++i) {
      uint32_t y;
      if constexpr (kEach == 2) y = k & 1 ? (r[i] & 0xffffu) | (uint32_t)v << 16 : (r[i] & 0xffff0000u) | v;
      else y = __float_as_uint(v);
      r[i] = i == k / kEach ? y : r[i];
    }
  }
};

// CHUNKS: of a row's piece for each thread.  LONG: lists of more than kListed biases.
template <class T, int CHUNKS, bool LONG>
__global__ __launch_bounds__(kLogitThreads, 8) void adjust_kernel(LogitArgs a) {
  typedef typename Logit<T>::E E;
  constexpr int kWords = kChunk * sizeof(E) / 16, kPiece = CHUNKS * kChunk * kLogitThreads;
  __shared__ __align__(16) uint32_t table[kPiece], touched[kPiece / 32];       // the words in use, as bits
  __shared__ __align__(16) int listed_token[kListed];
  __shared__ int listed_at[kListed], listed;
  __shared__ float listed_bias[kListed];
  __shared__ __align__(16) uint32_t named[LONG ? kPiece : 4];          // an entry's last place in the list and 1
  __shared__ double shared_inverse;
  const int tid = threadIdx.x;
  const int pieces = (a.vocab + kPiece - 1) / kPiece;
  const int64_t t = blockIdx.x / pieces;
  const int piece = (int)(blockIdx.x - t * pieces), V = a.vocab;
  const int s = owner_of(a.starts, a.seqs, t);
  // What there is of the sequence, in one go: a load in a branch of its own would be waited for before the next, and
  // these would be as many turns of latency.  What is not given is read from starts, and not used.
  const auto given = [&](const void *p) { return ((const uint32_t *)(p ? p : a.starts))[s]; };
  int64_t begin = a.starts[s], end = a.starts[s + 1];
  const int len = (int)given(a.lens), prompt_len = (int)given(a.prompt_lens);
  const float rep32 = __uint_as_float(given(a.repetition)), pres32 = __uint_as_float(given(a.presence));
  const float freq32 = __uint_as_float(given(a.frequency));
  begin = begin < 0 ? 0 : begin;
  end = end > a.rows ? a.rows : end;
  if (t < begin || t >= end) return;         // of no sequence

  // Strips of 512 entries are dealt to the pieces in turn: a text's common tokens lie close together.
  const auto entry_at = [&](int word) { return (int64_t)(word / kStrip * pieces + piece) * kStrip + word % kStrip; };
  const auto place = [&](int x) {            // where x's word is; -1: another piece's
    // below 2^21 strips: half a strip over a multiple is farther from it than the product is off
    const int strip = (int)((uint32_t)x / kStrip), mine = (int)(((float)strip + 0.5f) * a.pieces_inverse);
    return (uint32_t)x < (uint32_t)V && strip - __mul24(mine, pieces) == piece ? mine * kStrip + (x & (kStrip - 1)) : -1;
  };
  Held<E> u[CHUNKS];
  uint32_t mask_word[CHUNKS];
  const E *in = (const E *)a.logits + t * a.stride;
  E *out = (E *)a.out + t * a.out_stride;
  const uint32_t *mask = a.mask ? a.mask + t * a.mask_stride : nullptr;
  // The piece, its mask, the text's first tokens and the first biases on their way while the table is made.  No thread
  // has a way around any of these loads, which would be waited for at its end: past the last entry they read it again.
  const bool fast = a.whole && V >= kChunk;
  const auto start = [&](int c) { return entry_at((c * kLogitThreads + tid) * kChunk); };
  if (fast) {
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
      const int64_t x0 = start(c), last = (V - kChunk) / kChunk * kChunk;
#pragma unroll
      for (int k = 0; k < kWords; ++k) u[c].w[k] = ((const u32x4 *)(in + (x0 < last ? x0 : last)))[k];
    }
  }
  if (mask) {
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
      const int64_t x0 = start(c);
      mask_word[c] = mask[(x0 < V ? x0 : V - 1) >> 5];
    }
  }
  const bool rules = a.text || a.biases;
  const int32_t *text = a.text + s * a.text_stride;
  const int32_t *bias_tokens = a.bias_tokens + (int64_t)s * a.biases;
  const float *bias = a.bias + (int64_t)s * a.biases;
  const bool quads = a.text && ((uintptr_t)text & 15) == 0 && a.text_width >= 4;
  const int quarter = a.text_width & ~3;     // the text in fours, and the rest
  const auto four_at = [&](int i) { return *(const u32x4 *)(text + (i < quarter - 4 ? i : quarter - 4)); };
  u32x4 four = (u32x4){0, 0, 0, 0};
  if (quads) four = four_at(4 * tid);
  int first_token = -1;
  float first_bias = 0.0f;
  if (a.biases) {
    const int i = tid < a.biases ? tid : a.biases - 1;
    first_token = bias_tokens[i];
    first_bias = bias[i];
  }
  const int prompt = a.prompt_lens ? prompt_len : 0;
  int m = 0;                                 // tokens up to the row's own
  const double rep = a.repetition ? (double)rep32 : 1.0, pres = a.presence ? (double)pres32 : 0.0;
  const double freq = a.frequency ? (double)freq32 : 0.0;
  const auto touch = [&](int at) { atomicOr(&touched[at >> 5], 1u << (at & 31)); };
  const auto count = [&](int x, int i) {
    const int at = place(x);
    if (at < 0) return;
    if (i < prompt) atomicOr(&table[at], kInPrompt);
    else atomicAdd(&table[at], 1u);
    touch(at);
  };
  if (rules) {
    if (a.text) {
      const int64_t n = len - (end - t) + 1;
      m = (int)(n < 0 ? 0 : n < a.text_width ? n : a.text_width);
    }
    for (int i = tid * 4; i < kPiece; i += kLogitThreads * 4) {
      *(u32x4 *)(table + i) = (u32x4){0, 0, 0, 0};
      if (LONG) *(u32x4 *)(named + i) = (u32x4){0, 0, 0, 0};
    }
    for (int i = tid; i < kPiece / 32; i += kLogitThreads) touched[i] = 0;
    if (tid == 0) listed = 0;
    for (int i = tid; i < kListed; i += kLogitThreads) listed_token[i] = -1;
    __syncthreads();
    if (tid >= kLogitThreads - kWave) shared_inverse = 1.0 / rep;      // the last wave has the least of a short text
    int rest = 0;
    if (quads) {
      rest = quarter;
      const int w = m < quarter ? m : quarter;
      for (int from = 0; from < w; from += 4 * kLogitThreads) {
        const int i = from + 4 * tid;
        u32x4 next = four;
        if (from + 4 * kLogitThreads < w) next = four_at(i + 4 * kLogitThreads);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (i + k < w) count((int)four[k], i + k);
        four = next;
      }
    }
    for (int i = rest + tid; i < m; i += kLogitThreads) count(text[i], i);
    for (int i = tid; i < a.biases; i += kLogitThreads) {
      const int x = i == tid ? first_token : bias_tokens[i], word = place(x);
      if (word < 0) continue;
      atomicOr(&table[word], kBiased);
      touch(word);
      if (LONG) {
        atomicMax(&named[word], (uint32_t)i + 1u);
        continue;
      }
      const int at = atomicAdd(&listed, 1);
      listed_token[at] = x;
      listed_at[at] = i;
      listed_bias[at] = i == tid ? first_bias : bias[i];
    }
    __syncthreads();
  }
  // of equal biases the last in the list, whichever order they came to LDS in
  const int biases = listed;
  const auto bias_of = [&](int x, int word) {
    if (LONG) return (double)bias[named[word] - 1u];
    int last = -1;
    float v = 0.0f;
    for (int i = 0; i < biases; i += 4) {
      const u32x4 four = *(const u32x4 *)(listed_token + i);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if ((int)four[k] == x && listed_at[i + k] > last) {
          last = listed_at[i + k];
          v = listed_bias[i + k];
        }
    }
    return (double)v;
  };
  const double inverse = shared_inverse;
  // A logit by its entry's word, the word-th of the piece.
  const auto ruled = [&](E e, uint32_t w, int x, int word) {
    const uint32_t made = w & kMade;
    const double l = (double)Logit<T>::get(e);
    double q = l * inverse;                  // an exact quotient comes out exact
    const double exact = __builtin_fma(__builtin_fma(-q, rep, l), inverse, q);
    q = __builtin_fabs(q) < INFINITY && q != 0.0 ? exact : q;
    double z = w & (kInPrompt | kMade) ? l > 0.0 ? q : l * rep : l;
    z = made ? z - (freq * (double)made + pres) : z;
    if (w & kBiased) z += bias_of(x, word);
    return Logit<T>::put(z);
  };
  // the piece, masked
  const uint32_t none = sizeof(E) == 4 ? __float_as_uint(-INFINITY) : (uint32_t)Logit<T>::put(-(double)INFINITY) * 0x10001u;
#pragma unroll
  for (int c = 0; c < CHUNKS; ++c) {
    const int64_t x0 = start(c);
    if (x0 >= V) break;
    const uint32_t bits = mask ? mask_word[c] >> (x0 & 31) : 0xffu;
    const bool whole = fast && x0 + kChunk <= V;
    if (!whole) {
#pragma unroll
      for (int k = 0; k < kChunk; ++k) u[c].e[k] = x0 + k < V ? in[x0 + k] : E(0);
    }
    const int word = (c * kLogitThreads + tid) * kChunk;
    const uint32_t own = rules ? ((const uint8_t *)touched)[word / kChunk] & bits : 0u;
    // Few work-groups wait for the slowest lane, that of a text's common tokens, which lie together: the lanes' first
    // entries, then their second ones, without a branch in them (one row of 32,000 fp32 entries: 4.8 us of the GPU, 5.7
    // otherwise, 7.0 without a mask).  Many have more to do: each lane its own entries (157 rows: 24.4 us, 26 otherwise).
    if constexpr (CHUNKS == 1) {
      if (__any(own)) {
        uint32_t seen[kChunk];
#pragma unroll
        for (int k = 0; k < kChunk; k += 4) *(u32x4 *)(seen + k) = *(const u32x4 *)(table + word + k);
#pragma unroll
        for (int k = 0; k < kChunk; ++k) {
          const bool mine = (own >> k) & 1u;
          if (!__any(mine)) continue;
          const E y = ruled(u[c].e[k], mine ? seen[k] : 0u, (int)x0 + k, word + k);
          u[c].e[k] = mine ? y : u[c].e[k];
        }
      }
    } else {
      for (uint32_t left = own; left; left &= left - 1) {
        const int k = __ffs(left) - 1;
        u[c].put(k, ruled(u[c].at(k), table[word + k], (int)x0 + k, word + k));
      }
    }
    if (mask) {
      constexpr int kEach = 4 / sizeof(E);               // entries of 32 bits
#pragma unroll
      for (int w = 0; w < kChunk / kEach; ++w) {
        // a bit as all bits of its entry
        uint32_t stays = (uint32_t)__builtin_amdgcn_sbfe((int)bits, w * kEach, 1), other;
        if (kEach == 2) {
          other = (uint32_t)__builtin_amdgcn_sbfe((int)bits, w * kEach + 1, 1);
          stays = (stays & 0xffffu) | (other & 0xffff0000u);
        }
        uint32_t &x = u[c].r[w];
        x = (x & stays) | (none & ~stays);
      }
    }
    if (whole) {
#pragma unroll
      for (int k = 0; k < kWords; ++k) ((u32x4 *)(out + x0))[k] = u[c].w[k];
    } else {
#pragma unroll
      for (int k = 0; k < kChunk; ++k)
        if (x0 + k < V) out[x0 + k] = u[c].e[k];
    }
  }
}

template <class T, int CHUNKS>
void launch_chunks(const LogitArgs &a, dim3 grid, hipStream_t st) {
  if (a.biases > kListed) adjust_kernel<T, CHUNKS, true><<<grid, kLogitThreads, 0, st>>>(a);
  else adjust_kernel<T, CHUNKS, false><<<grid, kLogitThreads, 0, st>>>(a);
}
template <class T>
void launch_type(const LogitArgs &a, dim3 grid, hipStream_t st) {
  if (a.piece == kLogitPiece) launch_chunks<T, 2>(a, grid, st);
  else launch_chunks<T, 1>(a, grid, st);
}

}  // namespace

void launch_adjust_logits(const LogitArgs &a, int type, dim3 grid, hipStream_t st) {
  if (type == CT_BF16) launch_type<Bf16>(a, grid, st);
  else if (type == CT_F16) launch_type<F16>(a, grid, st);
  else launch_type<float>(a, grid, st);
}

}  // namespace kmi
