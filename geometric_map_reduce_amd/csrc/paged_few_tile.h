// paged_few_tile.h -- one tile of the few-rows attention (paged_few.h), a part of its kernel's body: the tile `tile` that
// has arrived in `f` (4-bit caches: at `stage`), and the loads of the one at `next`.
//
// It is included where it runs, in the tile loop of 16-bit and 8-bit caches and in the function that 4-bit caches call
// for each of a turn's two tiles.  As such a function it cost the others registers: e4m3, dim 96, 17 to 32 rows 257 in
// place of 240, and so one work-group a compute unit in place of two and other parts of a row's sums; with weights up
// to 6 spilled.  Times are the same to a percent (64 x 4,096 slots of 8 x 96, 32 rows: 164 us), HBM bounds them.
const int at = tile * kFewTile, j0 = blk + at;
if constexpr (E2M1) f.take_keys(stage);
f32x4 sc[NR][2];
#pragma unroll
for (int t = 0; t < 2; ++t) {
#pragma unroll
  for (int nr = 0; nr < NR; ++nr) sc[nr][t] = (f32x4){0, 0, 0, 0};
#pragma unroll
  for (int st = 0; st < F::kSteps; ++st) {
    const u32x4 kf = f.k_frag(t, st);
#pragma unroll
    for (int nr = 0; nr < NR; ++nr) sc[nr][t] = T::mfma16(kf, qf[nr][st], sc[nr][t]);
  }
}
if constexpr (E2M1) load_next(f, next);
else f.template load_k<FAR>(kbase, sh.off, next);
__builtin_amdgcn_sched_barrier(0);

const uint32_t there = present[tile];
const bool masked = there != 0xffffffffu || j0 + kFewTile - 1 > sp.first || (a.window > 0 && j0 <= last_pos - a.window);
if (masked) {
#pragma unroll
  for (int nr = 0; nr < NR; ++nr) {
    const int up = pos[nr] - j0;
    uint32_t own = first_bits(up + 1) & there;      // the row's slots, as bits
    if (a.window > 0) own &= ~first_bits(up + 1 - a.window);
    own >>= q4 * 4;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (!(own & (1u << ((i >> 2) * 16 + (i & 3))))) sc[nr][i >> 2][i & 3] = -INFINITY;
  }
}
u32x4 pf[NR], pr;          // p, and what its rounding left
#pragma unroll
for (int nr = 0; nr < NR; ++nr) {
  float z[8], top = -INFINITY;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    z[i] = sc[nr][i >> 2][i & 3] * c;
    top = fmaxf(top, z[i]);
  }
  if (SCORES) {
    const int r = 16 * nr + col;
    if (r < R) {
      // groups of four slots, a group's rows together
      float *at4 = scores + (((at >> 2) + q4) * a.score_rows + r) * 4;
      *(f32x4 *)at4 = (f32x4){z[0], z[1], z[2], z[3]};
      *(f32x4 *)(at4 + 16 * a.score_rows) = (f32x4){z[4], z[5], z[6], z[7]};
    }
  }
  if (__any(top > m_run[nr] + (kLazy + T::kShift))) {
    const float m_new = fmaxf(m_run[nr], xor_max(top) - T::kShift);
    const float alpha = m_new == -INFINITY ? 1.0f : fast_exp2(m_run[nr] - m_new);
    l_run[nr] *= alpha;
    m_run[nr] = m_new;
#pragma unroll
    for (int t = 0; t < F::kTiles; ++t) acc[nr][t] *= alpha;
  }
  const float m_use = m_run[nr] == -INFINITY ? 0.0f : m_run[nr];
  float p[8], sum = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    p[i] = fast_exp2(z[i] - m_use);
    sum += p[i];
  }
  l_run[nr] += sum;
#pragma unroll
  for (int u = 0; u < 4; ++u) pf[nr][u] = T::pack(p[2 * u], p[2 * u + 1]);
  if constexpr (kBoth) {
#pragma unroll
    for (int u = 0; u < 4; ++u)
      pr[u] = T::pack(p[2 * u] - T::lo(pf[nr][u]), p[2 * u + 1] - T::hi(pf[nr][u]));
  }
}
if constexpr (E2M1) f.take_staged(stage);
bool past = false;         // a block of the tile may hold an infinity or is a NaN
if constexpr (kBoth) {
  uint32_t power = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int n = 0; n < VPieces<D>::n; ++n) power = f.vp[i][n] > power ? f.vp[i][n] : power;
  past = __any(power > T::kE2m1Top);
}
if (masked || past) {
  // absent slots are zeros; non-finite values of slots that some rows see and others do
  // not wait for the end.  So do all where p's remainder is multiplied too: it is 0 or below it as often as above, and
  // an infinity times that is NaN or the other infinity
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int u = (i >> 2) * 16 + q4 * 4 + (i & 3), j = j0 + u;
    const bool keep = (there >> u) & 1u;
    const bool some = kBoth || j > sp.first || (a.window > 0 && j <= last_pos - a.window);
#pragma unroll
    for (int k = 0; k < F::kVRegs; ++k) {
      if (E2M1) {
        uint32_t &w = f.vr[i][k], &power = f.vp[i][k % VPieces<D>::n];
        w = keep ? w : 0u;
        power = keep ? power : 127u;
        if (some && power > T::kE2m1Top) {
          const uint32_t y = finite_codes<T>(w, power);
          odd |= y != w || power == 255u;       // 255: a NaN whatever the code
          w = y;
          power = power == 255u ? 127u : power;
        }
        continue;
      }
      const uint32_t x = keep ? f.vr[i][k] : 0u;
      const uint32_t y = some ? (E4M3 ? finite_bytes(x) : finite_halves<T>(x)) : x;
      odd |= y != x;
      f.vr[i][k] = y;
    }
  }
}
int t = 0;
#pragma unroll
for (int n = 0; n < VPieces<D>::n; ++n)
#pragma unroll
  for (int m = 0; m < VPieces<D>::w[n] / 2; ++m, t += 2) {
    u32x4 x, y;
    f.v_frags(n, m, x, y);
#pragma unroll
    for (int nr = 0; nr < NR; ++nr) {
      acc[nr][t] = T::mfma16(x, pf[nr], acc[nr][t]);
      acc[nr][t + 1] = T::mfma16(y, pf[nr], acc[nr][t + 1]);
      if constexpr (kBoth) {
        acc[nr][t] = T::mfma16(x, pr, acc[nr][t]);
        acc[nr][t + 1] = T::mfma16(y, pr, acc[nr][t + 1]);
      }
    }
  }
if constexpr (!E2M1) f.template load_v<FAR>(vbase, sh.off, next);
