// paged_join.hip -- the paged attention's launches, and the second passes of its many-rows form:
// joining the slot splits, and partial column sums into the slots' attention weights.
#include "paged.h"

namespace kmi {

// paged_few_*.hip and paged_many_*.hip
using FewLaunch = int(const AttendArgs &a, int dim, int row_tiles, int grid, int join_rows, hipStream_t st);
using ManyLaunch = void(const AttendArgs &a, int dim, bool sums, dim3 grid, hipStream_t st);
FewLaunch few_bf16, few_f16, few_bf16_e4m3, few_f16_e4m3, few_bf16_e2m1, few_f16_e2m1;
ManyLaunch many_bf16, many_f16, many_bf16_e4m3, many_f16_e4m3, many_bf16_e2m1, many_f16_e2m1;

namespace {

// out = sum_k 2^(m_k - M) o_k / sum_k 2^(m_k - M) l_k over the splits k under a running maximum M.
// `per_row` groups of dim / 4 threads share a row (one where the splits are few), splits in order
// within each, then the groups in order.
template <class T>
__global__ __launch_bounds__(kJoinThreads) void join_kernel(AttendArgs a, int per_row) {
  __shared__ f32x4 part[kJoinThreads];
  __shared__ float2 part_ml[kJoinThreads];
  const int D = a.c.dim, lanes = D / 4, tid = threadIdx.x;
  const int g = tid / lanes, d4 = tid - g * lanes, gr = g / per_row, gk = g - gr * per_row;
  const int rows_per = kJoinThreads / lanes / per_row;
  const int64_t rows = a.tokens * a.c.heads * a.group, row = (int64_t)blockIdx.x * rows_per + gr;
  const bool mine = gr < rows_per && row < rows;
  f32x4 acc = (f32x4){0, 0, 0, 0};
  float l = 0.0f, top = -INFINITY;
  const auto add = [&](float m, float y, f32x4 o) {
    if (!(y > 0.0f || y != y)) return;         // a split without a slot: its sums were not written
    const float m_new = fmaxf(top, m), x = fast_exp2(top - m_new), z = fast_exp2(m - m_new);
    l = l * x + y * z;
    acc = acc * x + o * z;
    top = m_new;
  };
  if (mine) {
    for (int k = gk; k < a.nsplit; k += 4 * per_row) {
      float2 x[4];
      f32x4 o[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int64_t at = (int64_t)(k + u * per_row < a.nsplit ? k + u * per_row : a.nsplit - 1) * rows + row;
        x[u] = a.part_ml[at];
        o[u] = *(const f32x4 *)(a.part_o + at * D + d4 * 4);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (k + u * per_row < a.nsplit) add(x[u].x, x[u].y, o[u]);
    }
  }
  if (per_row > 1) {
    part[tid] = acc;
    part_ml[tid] = make_float2(top, l);
    __syncthreads();
    if (mine && gk == 0)
      for (int k = 1; k < per_row; ++k) add(part_ml[tid + k * lanes].x, part_ml[tid + k * lanes].y, part[tid + k * lanes]);
  }
  if (!mine || gk != 0) return;
  const bool any = l > 0.0f || l != l;
  const float mul = any ? 1.0f / l : 0.0f;
  if (d4 == 0) a.lse[row] = any ? (top + __log2f(l)) * kLn2 : -INFINITY;
  // an absent row has zeros, not 0 * infinity
  const f32x4 o = any ? acc * mul : (f32x4){0, 0, 0, 0};
  *(u32x2 *)(a.out + (row * D + d4 * 4) * 2) = (u32x2){T::pack(o[0], o[1]), T::pack(o[2], o[3])};
}

__device__ __forceinline__ void put_weight(const AttendArgs &a, SlotPlace p, int h, float w) {
  if (p.page < 0) return;
  float *at = a.c.weights + ((int64_t)p.page * a.c.heads + h) * a.c.page.d + p.row;
  *at = a.decay != 0.0f ? a.decay * *at + w : w;
}

// Weights of the many-rows form from its row splits, in order.
__global__ __launch_bounds__(256) void sums_join_kernel(AttendArgs a) {
  const int H = a.c.heads;
  const int blocks = (a.max_len + 255) / 256;
  const int sh = blockIdx.x / blocks, s = sh / H, h = sh - s * H;
  const SeqSpan sp = seq_span(a.starts, a.c.lens, s, a.tokens, a.max_q, a.max_len);
  const int j = (blockIdx.x - sh * blocks) * 256 + threadIdx.x;
  if (j >= sp.n) return;
  float w = 0.0f;
  for (int k = 0; k < a.nrow; ++k) w += a.part_w[((int64_t)k * a.c.seqs * H + sh) * a.max_len + j];
  put_weight(a, slot_place(a.c, a.c.table + (int64_t)s * a.c.table_stride, (uint32_t)j), h, w);
}

}  // namespace

int launch_attend_few(const AttendArgs &a, int type, int bits, int dim, int row_tiles, int grid, int join_rows,
                      hipStream_t st) {
  FewLaunch *f = type == CT_BF16 ? (bits == 4 ? few_bf16_e2m1 : bits == 8 ? few_bf16_e4m3 : few_bf16)
                                 : (bits == 4 ? few_f16_e2m1 : bits == 8 ? few_f16_e4m3 : few_f16);
  return f(a, dim, row_tiles, grid, join_rows, st);
}

static ManyLaunch *many_of(int type, int bits) {
  return type == CT_BF16 ? (bits == 4 ? many_bf16_e2m1 : bits == 8 ? many_bf16_e4m3 : many_bf16)
                         : (bits == 4 ? many_f16_e2m1 : bits == 8 ? many_f16_e4m3 : many_f16);
}

void launch_attend_many(const AttendArgs &a, int type, int bits, int dim, dim3 grid, hipStream_t st) {
  many_of(type, bits)(a, dim, false, grid, st);
}

void launch_attend_sums(const AttendArgs &a, int type, int bits, int dim, dim3 grid, hipStream_t st) {
  many_of(type, bits)(a, dim, true, grid, st);
}

void launch_attend_join(const AttendArgs &a, int type, hipStream_t st) {
  const int per_row = join_per_row(a.c.dim, a.nsplit);
  const dim3 grid((unsigned)join_blocks(a.tokens * a.c.heads * a.group, a.c.dim, a.nsplit));
  if (type == CT_BF16) join_kernel<Bf16><<<grid, kJoinThreads, 0, st>>>(a, per_row);
  else join_kernel<F16><<<grid, kJoinThreads, 0, st>>>(a, per_row);
}

void launch_attend_sums_join(const AttendArgs &a, hipStream_t st) {
  const int64_t blocks = (a.max_len + 255) / 256;
  sums_join_kernel<<<dim3((unsigned)(blocks * a.c.seqs * a.c.heads)), 256, 0, st>>>(a);
}

}  // namespace kmi
