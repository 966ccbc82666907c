// paged_append_rotary.hip -- queries and keys turned to their positions, keys and values into their slots.
//
//   q_out[t, g] = R(p) q[t, g],   pages[slot of t][h] = R(p) k[t, h], v[t, h],   p = positions[t] or the slot's number
//
// where R turns the pairs of columns by p freqs[i] (rotary.hip).  Each element is read once from HBM (a pair's
// other column comes again by way of the caches) and written once.
//
// A work-group has up to four tokens: a wave finds a token's sequence and slot, then the threads compute the
// tokens' cosines and sines into LDS, in 64 bits, then each takes eight columns of a head at a time.  Queries and
// 16-bit keys are turned in 32 bits.  Keys that go into 8 or 4 bits are turned in 64: at 2^-24 some of every
// million would be decided wrongly at the borders between held values.
//
// Memory bounds a prompt: 16,384 tokens of 32 + 8 heads of 128 into 4 bits take 79 us (353 MB, 4.5 TB/s); cosines and
// sines held in 32 bits for the queries as well changed nothing, the next items' loads ahead of this one's arithmetic
// cost registers and 16 us.  1,200 tokens of nine sequences take 13 us, a chain: the sequence's number, its length, the
// table's entry, then the angles, then three turns of loads; one token of 64 sequences 3.9 us.
#include "step.h"

namespace kmi {
namespace {

// Eight columns from d on of the row at x, turned.  R: the type of the arithmetic.
template <class T, class R>
__device__ __forceinline__ void turn8(const char *x, int d, const double2 *cs, int n, bool interleaved, R (&out)[8]) {
  float own[8];
  widen8<T>(*(const u32x4 *)(x + d * 2), own);
#pragma unroll
  for (int u = 0; u < 8; ++u) out[u] = (R)own[u];
  if (d >= 2 * n) return;
  if (interleaved) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (d / 2 + k >= n) continue;
      const double2 by = cs[d / 2 + k];
      const R c = (R)by.x, s = (R)by.y, a = (R)own[2 * k], b = (R)own[2 * k + 1];
      out[2 * k] = fma(a, c, b * -s);
      out[2 * k + 1] = fma(b, c, a * s);
    }
  } else if (n % 8 == 0) {
    const bool second = d >= n;
    const int i = second ? d - n : d;
    float other[8];
    widen8<T>(*(const u32x4 *)(x + (second ? d - n : d + n) * 2), other);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const double2 by = cs[i + u];
      const R c = (R)by.x, s = second ? (R)by.y : -(R)by.y;
      out[u] = fma((R)own[u], c, (R)other[u] * s);
    }
  } else {
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      if (d + u >= 2 * n) continue;
      const bool second = d + u >= n;
      const int i = second ? d + u - n : d + u;
      const float other = T::lo(*(const uint16_t *)(x + (second ? i : i + n) * 2));
      const double2 by = cs[i];
      const R c = (R)by.x, s = second ? (R)by.y : -(R)by.y;
      out[u] = fma((R)own[u], c, (R)other * s);
    }
  }
}

template <class T>
__device__ __forceinline__ u32x4 pack8(const float (&x)[8]) {
  return (u32x4){T::pack(held(x[0]), held(x[1])), T::pack(held(x[2]), held(x[3])), T::pack(held(x[4]), held(x[5])),
                 T::pack(held(x[6]), held(x[7]))};
}

template <class T, int BITS>
__global__ __launch_bounds__(kTurnThreads) void append_rotary_kernel(AppendRotaryArgs a) {
  extern __shared__ double2 turned[];                   // [tokens of the work-group][pairs]
  __shared__ SlotPlace place[kTurnTokens];
  __shared__ int position[kTurnTokens];
  __shared__ bool live[kTurnTokens];                    // in a sequence
  const int tid = threadIdx.x, lane = tid & (kWave - 1), n = a.r.pairs, D = a.c.dim, H = a.c.heads;
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int64_t t0 = (int64_t)blockIdx.x * a.tokens_wg;
  const int tokens = a.tokens - t0 < a.tokens_wg ? (int)(a.tokens - t0) : a.tokens_wg;
  static_assert(kTurnTokens <= kTurnThreads / kWave, "a wave for each token");
  if (wave < tokens) {
    const int64_t t = t0 + wave;
    const int s = owner_of(a.starts, a.c.seqs, t);
    const SeqSpan sp = seq_span(a.starts, a.c.lens, s, a.tokens, 0x7fffffff, 0x7fffffff);
    const bool in = t >= sp.t0 && t < sp.t0 + sp.m;
    const int64_t j = sp.first + (t - sp.t0);           // below 0 where there are fewer slots than new tokens
    SlotPlace p{-1, 0};
    if (in && j >= 0) p = slot_place(a.c, a.c.table + (int64_t)s * a.c.table_stride, (uint32_t)j);
    if (lane == 0) {
      place[wave] = p;
      live[wave] = in;
      position[wave] = a.positions ? a.positions[t] : (int)j;
    }
  }
  __syncthreads();
  for (int i = tid; i < tokens * n; i += kTurnThreads) {
    const int t = i / n;
    turned[i] = rotation(a.r, position[t], i - t * n);
  }
  __syncthreads();
  const int per = (a.heads + 2 * H) * (D / 8);
  const int step = gridDim.y * kTurnThreads;
  for (int id = blockIdx.y * kTurnThreads + tid; id < tokens * per; id += step) {
    const int t = (int)fast_div(a.items_div, (uint32_t)id), e = id - t * per;
    const int head = (int)fast_div(a.dim_div, (uint32_t)e), d = (e - head * (D / 8)) * 8;
    if (!live[t]) continue;
    const double2 *cs = turned + t * n;
    if (head < a.heads) {
      float x[8];
      turn8<T>(a.q + (t0 + t) * a.q_stride + (int64_t)head * D * 2, d, cs, n, a.r.interleaved, x);
      *(u32x4 *)(a.q_out + (t0 + t) * a.q_out_stride + ((int64_t)head * D + d) * 2) = pack8<T>(x);
      continue;
    }
    const SlotPlace p = place[t];
    if (p.page < 0) continue;
    const bool key = head < a.heads + H;
    const int h = head - a.heads - (key ? 0 : H);
    const char *x = (key ? a.k + (t0 + t) * a.k_stride : a.v + (t0 + t) * a.v_stride) + (int64_t)h * D * 2;
    char *to = (key ? a.c.k : a.c.v) + place_offset(a.c, p) + (int64_t)h * a.c.head_stride + d * BITS / 8;
    if (a.c.weights && key && d == 0) a.c.weights[((int64_t)p.page * H + h) * a.c.page.d + p.row] = 0.0f;
    if constexpr (BITS == 16) {
      if (!key) {
        *(u32x4 *)to = *(const u32x4 *)(x + d * 2);
        continue;
      }
      float y[8];
      turn8<T>(x, d, cs, n, a.r.interleaved, y);
      *(u32x4 *)to = pack8<T>(y);
    } else {
      float y[8];
      if (key) {
        double z[8];
        turn8<T>(x, d, cs, n, a.r.interleaved, z);
        if (BITS == 8) {
          const double s = (double)a.c.k_scale[h], inverse = 1.0 / s;
#pragma unroll
          for (int u = 0; u < 8; ++u) y[u] = e4m3_of(z[u], s, inverse);
        } else {
#pragma unroll
          for (int u = 0; u < 8; ++u) y[u] = round_to_odd(z[u]);
        }
      } else {
        widen8<T>(*(const u32x4 *)(x + d * 2), y);
        if (BITS == 8) {
          const float s = a.c.v_scale[h];
#pragma unroll
          for (int u = 0; u < 8; ++u) y[u] = e4m3_quotient(y[u], s);
        }
      }
      if (BITS == 8) {
        *(u32x2 *)to = pack_e4m3(y);
      } else {
        // the four threads of a block go the same way
        uint32_t power;
        *(uint32_t *)to = to_e2m1(y, T::kE2m1Top, &power);
        if (d % kPowerBlock == 0)
          (key ? a.c.k_power : a.c.v_power)[(uint64_t)place_number(a.c, p, h) * (D / kPowerBlock) + d / kPowerBlock] = (uint8_t)power;
      }
    }
  }
}

template <class T>
void launch_bits(const AppendRotaryArgs &a, int bits, dim3 grid, size_t lds, hipStream_t st) {
  if (bits == 4) append_rotary_kernel<T, 4><<<grid, kTurnThreads, lds, st>>>(a);
  else if (bits == 8) append_rotary_kernel<T, 8><<<grid, kTurnThreads, lds, st>>>(a);
  else append_rotary_kernel<T, 16><<<grid, kTurnThreads, lds, st>>>(a);
}

}  // namespace

void launch_append_rotary(const AppendRotaryArgs &a, int type, int bits, dim3 grid, hipStream_t st) {
  const size_t lds = (size_t)a.tokens_wg * a.r.pairs * sizeof(double2);
  if (type == CT_BF16) launch_bits<Bf16>(a, bits, grid, lds, st);
  else launch_bits<F16>(a, bits, grid, lds, st);
}

}  // namespace kmi
