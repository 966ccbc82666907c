// step.h -- launch arguments of the operators around the paged cache: rotary positions, the append that
// rotates, reading slots back, and the adjustment of logits.
#pragma once

#include <type_traits>

#include "paged.h"
#include "rotary.h"

namespace kmi {

constexpr int kRotaryThreads = 256;
struct RotaryArgs {
  const void *x;
  void *out;
  int64_t x_stride, out_stride;      // elements from token to token
  const int32_t *positions;
  RotaryView r;
  int64_t tokens;
  int32_t heads, dim;
  int32_t tokens_wg;                 // tokens of a work-group
  int32_t pieces;                    // of a head: pairs / V that turn, then those that are copied
  FastDiv pairs_div, pieces_div, heads_div;
};

constexpr int kTurnThreads = 256;
constexpr int kTurnTokens = 4;       // tokens of a work-group of the rotating append at most
struct AppendRotaryArgs {
  CacheView c;
  const char *q, *k, *v;
  char *q_out;
  int64_t q_stride, k_stride, v_stride, q_out_stride;     // bytes from token to token
  const int32_t *starts, *positions;
  RotaryView r;
  int64_t tokens;
  int32_t heads;                     // of q
  int32_t tokens_wg;
  FastDiv items_div, dim_div;        // 8-column pieces of a token's q, k and v, and of a head
};

struct ReadArgs {
  CacheView c;
  char *k, *v;
  int64_t k_stride, v_stride;        // bytes from token to token
  const int32_t *starts;
  int64_t tokens;
};

struct LogitArgs {
  const void *logits;
  void *out;
  int64_t stride, out_stride;        // elements from row to row
  int64_t rows;
  int32_t vocab, piece;              // vocabulary entries of a work-group
  const int32_t *starts, *text, *lens, *prompt_lens;
  int64_t text_stride;
  const float *repetition, *presence, *frequency;
  const int32_t *bias_tokens;
  const float *bias;
  const uint32_t *mask;
  int64_t mask_stride;
  int32_t seqs, text_width, biases;
  float pieces_inverse;
  bool whole;                        // rows of logits and out start on 16 bytes
};
constexpr int kLogitThreads = 512;
constexpr int kLogitPiece = 8192;    // vocabulary entries of a work-group, or half of them

void launch_rotary(const RotaryArgs &a, int type, int piece, dim3 grid, hipStream_t st);
void launch_append_rotary(const AppendRotaryArgs &a, int type, int bits, dim3 grid, hipStream_t st);
void launch_read(const ReadArgs &a, int type, int bits, hipStream_t st);
void launch_adjust_logits(const LogitArgs &a, int type, dim3 grid, hipStream_t st);

// ---------------------------------------------------------------- device helpers

// The sequence that token t belongs to, the last s with starts[s] <= t, found by a wave together: 64 bounds at a
// time, so that up to 64 sequences take one load.  0 where there is none.
__device__ __forceinline__ int owner_of(const int32_t *starts, int seqs, int64_t t) {
  const int lane = threadIdx.x & (kWave - 1);
  int lo = 0, n = seqs;                       // it is among lo .. lo + n - 1
  while (n > 1) {
    const int step = (n + kWave - 1) / kWave, s = lo + lane * step;
    const bool le = lane * step < n && starts[s] <= t;
    const uint64_t who = __ballot(le);
    const int last = who ? 63 - __clzll((long long)who) : 0;
    lo += last * step;
    n = n - last * step < step ? n - last * step : step;
  }
  return lo;
}

// x as it is in 32 bits: no instruction that rounds a multiply-add straight to 16 bits takes x's place, which the
// compiler uses in one loop and not in the next.
__device__ __forceinline__ float held(float x) {
  asm("" : "+v"(x));
  return x;
}

// x rounded to 32 bits towards an odd last place where it is not exact: what is rounded to far fewer bits
// after that comes out as if from x itself.
__device__ __forceinline__ float round_to_odd(double x) {
  float f = (float)x;
  const double d = (double)f;
  if (d == x || x != x) return f;
  uint32_t b = __float_as_uint(f);
  if (__builtin_fabs(d) > __builtin_fabs(x)) --b;       // towards zero first
  return __uint_as_float(b | 1u);
}

// What e4m3 of x / s is rounded from: IEEE division, cut to the largest finite value, NaN kept.
__device__ __forceinline__ float e4m3_quotient(float x, float s) {
  const float q = x / s;
  return q != q ? q : fminf(fmaxf(q, -448.0f), 448.0f);
}
// The same of a 64-bit x, so that e4m3 comes out nearest to the quotient itself; inverse: 1 / s.
__device__ __forceinline__ float e4m3_of(double x, double s, double inverse) {
  double q = x * inverse;
  const double left = __builtin_fma(-q, s, x);          // exact quotients come out exact
  if (__builtin_fabs(q) < INFINITY && q != 0.0) q = __builtin_fma(left, inverse, q);     // 0 and by an infinite s as it is
  const float f = round_to_odd(q);
  return f != f ? f : fminf(fmaxf(f, -448.0f), 448.0f);
}

// The power of a block of e2m1 codes from the largest magnitude's 32 bits: the least under which it does not
// round past 6, that is, stays below 7.  With m the power of two of the magnitude, 2^(m - 2), or 2^(m - 1) from
// 1.75 2^m on.  255 for a NaN or an infinity.
__device__ __forceinline__ uint32_t block_power(uint32_t most, uint32_t top) {
  if (most >= 0x7f800000u) return 255u;
  const int b = (int)((most + 0x00200000u) >> 23) - 2;
  return b < 0 ? 0u : ((uint32_t)b > top ? top : (uint32_t)b);
}
// Eight values under a power as e2m1 codes, to nearest, halfway to the even code, cut to +-6.
__device__ __forceinline__ uint32_t e2m1_codes(const float (&x)[8], uint32_t power) {
  const float s = __uint_as_float(power << 23);        // the instruction takes the power from the exponent bits
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[0], x[1], s, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[2], x[3], s, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[4], x[5], s, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[6], x[7], s, 3);
  return power == 255u ? 0u : w;
}
// Eight columns of a block whose other columns are in the three lanes beside (lane / 4 alike): its power, which
// all four get, and the codes.
__device__ __forceinline__ uint32_t to_e2m1(const float (&x)[8], uint32_t top, uint32_t *power) {
  uint32_t most = 0;
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const uint32_t b = __float_as_uint(x[u]) & 0x7fffffffu;
    most = b > most ? b : most;
  }
  // quad permutations 1 0 3 2 and 2 3 0 1
  const uint32_t a = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)most, 0xb1, 0xf, 0xf, true);
  most = a > most ? a : most;
  const uint32_t b = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)most, 0x4e, 0xf, 0xf, true);
  most = b > most ? b : most;
  *power = block_power(most, top);
  return e2m1_codes(x, *power);
}

// Eight floats as e4m3.
__device__ __forceinline__ u32x2 pack_e4m3(const float (&x)[8]) {
  u32x2 w;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    int p = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * i], x[4 * i + 1], 0, false);
    w[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(x[4 * i + 2], x[4 * i + 3], p, true);
  }
  return w;
}

// Eight 16-bit values as floats.
template <class T>
__device__ __forceinline__ void widen8(u32x4 w, float (&x)[8]) {
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    x[2 * u] = T::lo(w[u]);
    x[2 * u + 1] = T::hi(w[u]);
  }
}

}  // namespace kmi
