// paged_join.hip -- the paged attention's launches, and the second passes of its many-rows form:
// joining the slot splits, and partial column sums into the slots' attention weights.
#include "paged.h"

namespace kmi {

// paged_few_*.hip and paged_many_*.hip
int few_bf16(const AttendArgs &a, int dim, int row_tiles, int grid, int join_rows, hipStream_t st);
int few_f16(const AttendArgs &a, int dim, int row_tiles, int grid, int join_rows, hipStream_t st);
int few_bf16_e4m3(const AttendArgs &a, int dim, int row_tiles, int grid, int join_rows, hipStream_t st);
int few_f16_e4m3(const AttendArgs &a, int dim, int row_tiles, int grid, int join_rows, hipStream_t st);
void many_bf16(const AttendArgs &a, int dim, bool sums, dim3 grid, hipStream_t st);
void many_f16(const AttendArgs &a, int dim, bool sums, dim3 grid, hipStream_t st);
void many_bf16_e4m3(const AttendArgs &a, int dim, bool sums, dim3 grid, hipStream_t st);
void many_f16_e4m3(const AttendArgs &a, int dim, bool sums, dim3 grid, hipStream_t st);

namespace {

constexpr int kJoinThreads = 256;

// One work-group per row: out = sum_k 2^(m_k - M) o_k / sum_k 2^(m_k - M) l_k, splits in order
// within each of the groups of dim / 4 threads, then the groups in order.
template <class T>
__global__ __launch_bounds__(kJoinThreads) void join_kernel(AttendArgs a) {
  __shared__ f32x4 part[kJoinThreads];
  __shared__ float red[kJoinThreads / kWave];
  const int D = a.c.dim, lanes = D / 4, groups = kJoinThreads / lanes, tid = threadIdx.x;
  const int64_t rows = a.tokens * a.c.heads * a.group, row = blockIdx.x;
  const float2 *ml = a.part_ml + row;
  float top = -INFINITY;
  for (int k = tid; k < a.nsplit; k += kJoinThreads) top = fmaxf(top, ml[(int64_t)k * rows].x);
  top = block_max(top, red);
  const float use = top == -INFINITY ? 0.0f : top;
  const int g = tid / lanes, d4 = tid - g * lanes;
  f32x4 acc = (f32x4){0, 0, 0, 0};
  float l = 0.0f;
  if (g < groups) {
    for (int k = g; k < a.nsplit; k += groups) {
      const float2 x = ml[(int64_t)k * rows];
      if (!(x.y > 0.0f || x.y != x.y)) continue;
      const float w = fast_exp2(x.x - use);
      l += w * x.y;
      acc += w * *(const f32x4 *)(a.part_o + ((int64_t)k * rows + row) * D + d4 * 4);
    }
  }
  // every group needs all groups' l: it travels with the columns
  __shared__ float part_l[kJoinThreads];
  part[tid] = acc;
  part_l[tid] = l;
  __syncthreads();
  if (g != 0) return;
  for (int k = 1; k < groups; ++k) {
    acc += part[k * lanes + d4];
    l += part_l[k * lanes + d4];
  }
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

int launch_attend_few(const AttendArgs &a, int type, bool e4m3, int dim, int row_tiles, int grid, int join_rows,
                      hipStream_t st) {
  if (type == CT_BF16) return (e4m3 ? few_bf16_e4m3 : few_bf16)(a, dim, row_tiles, grid, join_rows, st);
  return (e4m3 ? few_f16_e4m3 : few_f16)(a, dim, row_tiles, grid, join_rows, st);
}

void launch_attend_many(const AttendArgs &a, int type, bool e4m3, int dim, dim3 grid, hipStream_t st) {
  if (type == CT_BF16) (e4m3 ? many_bf16_e4m3 : many_bf16)(a, dim, false, grid, st);
  else (e4m3 ? many_f16_e4m3 : many_f16)(a, dim, false, grid, st);
}

void launch_attend_sums(const AttendArgs &a, int type, bool e4m3, int dim, dim3 grid, hipStream_t st) {
  if (type == CT_BF16) (e4m3 ? many_bf16_e4m3 : many_bf16)(a, dim, true, grid, st);
  else (e4m3 ? many_f16_e4m3 : many_f16)(a, dim, true, grid, st);
}

void launch_attend_join(const AttendArgs &a, int type, hipStream_t st) {
  const dim3 grid((unsigned)(a.tokens * a.c.heads * a.group));
  if (type == CT_BF16) join_kernel<Bf16><<<grid, kJoinThreads, 0, st>>>(a);
  else join_kernel<F16><<<grid, kJoinThreads, 0, st>>>(a);
}

void launch_attend_sums_join(const AttendArgs &a, hipStream_t st) {
  const int64_t blocks = (a.max_len + 255) / 256;
  sums_join_kernel<<<dim3((unsigned)(blocks * a.c.seqs * a.c.heads)), 256, 0, st>>>(a);
}

}  // namespace kmi
