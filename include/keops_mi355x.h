/*
 * keops_mi355x.h -- C ABI of the MI355X (gfx950) Gaussian map-reduce engine.
 *
 * The engine evaluates reductions over a symbolic matrix M_ij = F(x_i, y_j)
 * that is never stored: coefficients are computed on the fly, tile by tile,
 * with memory linear in M + N.  Sources (web pages about the KeOps library):
 *
 *  [KO-GPU]  "Kernel Operations on the GPU, with Autodiff, without Memory
 *            Overflows" (paper summary page): §1 "Target operation" (the
 *            Gaussian kernel product a_i = sum_j k(x_i, y_j) b_j, x_i, y_j in
 *            R^D, Gaussian k of deviation sigma > 0, M and N up to a billion);
 *            §2 "Generic reduction framework" (sum, max, argmin, log-sum-exp
 *            reductions of formulas over i- and j-variables), "Performance and
 *            differentiation" (argKmin; autodiff); §4 (D <= 100).
 *  [README]  KeOps README: "symbolic matrices" paragraph (c) (formula
 *            evaluated on the fly on data arrays x_i, y_j); PyTorch example
 *            (D_ij = sum of squared differences, K_ij = exp(-D_ij), .sum(),
 *            .logsumexp(), .argmin(), grad of (a**2).sum()).
 *  [ISSUE]   GitHub issue "Transparent interface for billion-scale matrices":
 *            an output parameter so that the user allocates the result
 *            tensor, and calls made without holding the Python lock.
 *
 * Common conventions for every entry point
 * ----------------------------------------
 *  Memory:    every array pointer is a DEVICE pointer on the HIP device that is
 *             current on the calling thread.  Arrays are dense, row-major,
 *             fp32 (indices int64), at least 4-byte aligned.
 *  Ownership: the caller allocates every input and output ([ISSUE], item 1).
 *             The library keeps no reference after returning, except through
 *             work queued on `stream`; the caller keeps the buffers alive
 *             until the stream has passed that work.  Outputs must not overlap
 *             inputs.  Split-j workspace belongs to the library: one device
 *             buffer per (device, stream), allocated on first need, grown
 *             when a call needs more, and reused in stream order by later
 *             calls on that stream, so that a call allocates nothing once
 *             its stream has seen a call of its size.  A buffer is freed
 *             (with hipFree) when it grows, when more than 32 are held, or
 *             when KEOPS_OPT_WS_CACHE is set to 2.  Destroy a stream only
 *             after its calls' work has completed: a stream created later
 *             may reuse the handle, and with it the buffer.
 *  Stream:    `stream` is a hipStream_t passed as void* (NULL = the default
 *             stream).  Calls only enqueue work and never synchronise; kernel
 *             faults surface at the caller's next synchronisation.
 *  Threads:   reentrant; may be called concurrently from several host
 *             threads on different streams.  Calls running concurrently on
 *             one GPU do not share memory.
 *  Errors:    0 = KEOPS_OK, negative = error (see below); no exception ever
 *             crosses the ABI, and on an error nothing has been enqueued (but after
 *             KEOPS_ERR_HIP, where some of a call's launches may have been).
 *  Sizes:     M = 0 is a no-op.  N = 0: sums and gradients are 0, LogSumExp
 *             is -inf; K-min needs 1 <= K <= N.
 *  Supported: D in 1..8, 16, 32, 50, 64, 100; E in 1..4; K in 1..16 or 32.
 *             Other values return KEOPS_ERR_UNSUPPORTED.
 *  Kernel:    k(x, y) = exp(-|x - y|^2 / sigma^2)   (sigma finite, > 0)
 *             (sigma = 1 is the README's exp(-D_ij)).
 */
#ifndef KEOPS_MI355X_H
#define KEOPS_MI355X_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define KEOPS_OK 0
#define KEOPS_ERR_INVALID_ARG (-1)  /* null pointer with non-zero size, negative size,
                                       sigma not finite or <= 0, K > N, overlap  */
#define KEOPS_ERR_UNSUPPORTED (-2)  /* D, E or K outside the compiled set; N >= 2^31 for K-min */
#define KEOPS_ERR_ALLOC (-3)        /* workspace allocation failed                 */
#define KEOPS_ERR_HIP (-4)          /* a HIP call or kernel launch failed          */
#define KEOPS_ERR_SCRATCH (-5)      /* keops_gauss_sum_noalloc: the call needs more device
                                       scratch than the library holds                 */

/*
 * Gaussian kernel sum ([KO-GPU] §1 "Target operation"; [README] K_ij.sum(dim=1)):
 *   out[i, e] = sum_j exp(-|x_i - y_j|^2 / sigma^2) * b[j, e]
 * x: [M, D], y: [N, D], b: [N, E], out: [M, E].
 */
int keops_gauss_sum(const float *x, const float *y, const float *b,
                    int64_t M, int64_t N, int32_t D, int32_t E, float sigma,
                    float *out, void *stream);

/*
 * keops_gauss_sum without any allocation, for callers that cannot allocate device
 * memory during the call: code under HIP graph capture, tight serving loops, and
 * harnesses that forbid hipMalloc.  Arguments, layouts, results and errors are those
 * of keops_gauss_sum (the same kernels run); the difference is the workspace.  Instead
 * of stream-ordered allocations, the split-j partial results (and, at D >= 32, one
 * form flag per 256 rows) go to a fixed 64 MiB device array inside the library, one
 * copy per GPU, allocated when the library's code is first loaded on that GPU and
 * held until the process ends.  When the partials of the usual launch plan do not
 * fit, the call uses fewer j-splits (at the fewest, none: then no scratch is used),
 * which changes only the fp32 rounding order.  KEOPS_ERR_SCRATCH: the form flags
 * alone exceed the array (D >= 32 with M above about 4e9 rows); nothing is enqueued.
 * Every call on one GPU uses that GPU's same array, which keeps the last call's
 * contents: calls that overlap in time on one GPU (different streams or threads,
 * not ordered by the caller) race on it and give undefined results.  Nothing in the
 * array needs to start at zero.
 */
int keops_gauss_sum_noalloc(const float *x, const float *y, const float *b,
                            int64_t M, int64_t N, int32_t D, int32_t E, float sigma,
                            float *out, void *stream);

/*
 * LogSumExp reduction ([KO-GPU] §2 reductions list; [README] .logsumexp()):
 *   out[i, e] = log sum_j exp(-|x_i - y_j|^2 / sigma^2 + b[j, e])
 * b enters additively in the exponent.  Shapes as keops_gauss_sum.
 */
int keops_gauss_lse(const float *x, const float *y, const float *b,
                    int64_t M, int64_t N, int32_t D, int32_t E, float sigma,
                    float *out, void *stream);

/*
 * Max / ArgMax and Min / ArgMin reductions of the kernel product ([KO-GPU] §2
 * reductions list; [README] feature list "Sum, LogSumExp, Min, Max but also
 * ArgMin, ArgMax"):
 *   keops_gauss_max: out[i, e] = max_j K_ij b[j, e],  out_idx[i, e] = its j
 *   keops_gauss_min: out[i, e] = min_j K_ij b[j, e],  out_idx[i, e] = its j
 * with K_ij = exp(-|x_i - y_j|^2/sigma^2); among equal values the smaller j is
 * returned.  out: [M, E] fp32; out_idx: [M, E] int64, 8-byte aligned.  The
 * values are compared in fp32 as computed (K to about 1e-6 relative), so two
 * j whose products differ by less than that may be returned either way.
 * N = 0 gives -inf (max) or +inf (min) and index -1; NaN products never win.
 * Requires N < 2^31.
 */
int keops_gauss_max(const float *x, const float *y, const float *b, int64_t M, int64_t N, int32_t D, int32_t E,
                    float sigma, float *out, int64_t *out_idx, void *stream);
int keops_gauss_min(const float *x, const float *y, const float *b, int64_t M, int64_t N, int32_t D, int32_t E,
                    float sigma, float *out, int64_t *out_idx, void *stream);

/*
 * Laplacian kernel sum ([README] feature list: a wide range of formulas,
 * beyond the Gaussian kernel):
 *   out[i, e] = sum_j exp(-|x_i - y_j| / sigma) b[j, e],  |.| the Euclidean norm.
 * Shapes, conventions and errors as keops_gauss_sum.  Computed from raw
 * differences (never the expanded distance, whose rounding near x = y would
 * reach the square root).
 */
int keops_laplace_sum(const float *x, const float *y, const float *b, int64_t M, int64_t N, int32_t D, int32_t E,
                      float sigma, float *out, void *stream);

/*
 * Gradient of the kernel sum with respect to x ([KO-GPU] §2 "Performance and
 * differentiation"; [README] torch.autograd.grad((a_i ** 2).sum(), [x])), as
 * the vector-Jacobian product with the cotangent g = dL/da:
 *   out[i, d] = sum_j (-2/sigma^2) exp(-|x_i-y_j|^2/sigma^2) <g_i, b_j> (x[i,d] - y[j,d])
 * g: [M, E]; out: [M, D].  For L = sum_i |a_i|^2 pass g = 2a.
 */
int keops_gauss_grad_x(const float *x, const float *y, const float *b, const float *g,
                       int64_t M, int64_t N, int32_t D, int32_t E, float sigma,
                       float *out, void *stream);

/*
 * Gradients of L = sum_ie g_ie a_ie with respect to the other two inputs of
 * the kernel sum ([KO-GPU] §2 "Performance and differentiation": every input
 * of a reduction is differentiable).  Both are reductions over the rows i,
 * one output per point y_j (the transposed map-reduce):
 *   keops_gauss_grad_y:  out[j, d] = sum_i (2/sigma^2) K_ij <g_i, b_j> (x[i,d] - y[j,d])   out: [N, D]
 *   keops_gauss_grad_b:  out[j, e] = sum_i K_ij g[i, e]                                    out: [N, E]
 * with K_ij = exp(-|x_i - y_j|^2/sigma^2), x: [M, D], y: [N, D], b: [N, E],
 * g: [M, E] (dL/da).  Sizes: N = 0 is a no-op; M = 0 writes zeros.  The rest
 * of the conventions (pointers, ownership, stream, errors) are those above;
 * out must not overlap any input.
 */
int keops_gauss_grad_y(const float *x, const float *y, const float *b, const float *g,
                       int64_t M, int64_t N, int32_t D, int32_t E, float sigma,
                       float *out, void *stream);
int keops_gauss_grad_b(const float *x, const float *y, const float *g,
                       int64_t M, int64_t N, int32_t D, int32_t E, float sigma,
                       float *out, void *stream);

/*
 * Block-sparse reductions ([KO-GPU] §3 "Applications": cluster-wise
 * block-sparsity for large kernel linear systems, §4: the block-sparse
 * truncation rule; [README] feature list: an interface for block-sparse
 * strategies).  Only the kept pairs (i, j) enter the reduction; they are given
 * as ranges over rows and points, typically of points sorted by cluster:
 *   ranges_i    [nri][2]  row range c = [ranges_i[c][0], ranges_i[c][1]); row
 *                         ranges must not overlap;
 *   slices_i    [nri]     end (exclusive) in redranges_j of row range c's j
 *                         ranges, non-decreasing; they start at slices_i[c-1]
 *                         (0 for c = 0);
 *   redranges_j [nrj][2]  j range k = [redranges_j[k][0], redranges_j[k][1])
 *                         inside [0, N).
 * Row i in row range c reduces over the j of its ranges, in the listed order
 * (a j listed twice counts twice); rows in no row range get the empty
 * reduction (0, or -inf for LogSumExp).  The three arrays are HOST arrays of
 * int64 (the library validates them and plans the launch on the host, then
 * copies what the kernels need); x, y, b, g, out are device arrays as above.
 * These calls synchronise `stream` once, after that copy.  Any invalid range
 * (out of bounds, overlapping row ranges, decreasing slices) returns
 * KEOPS_ERR_INVALID_ARG before any device work.
 *   keops_gauss_sum_ranges:    out [M, E] as keops_gauss_sum over the kept pairs
 *   keops_gauss_lse_ranges:    out [M, E] as keops_gauss_lse over the kept pairs
 *   keops_gauss_grad_x_ranges: out [M, D] as keops_gauss_grad_x over the kept pairs
 */
int keops_gauss_sum_ranges(const float *x, const float *y, const float *b, int64_t M, int64_t N, int32_t D,
                           int32_t E, float sigma, const int64_t *ranges_i, int64_t nri, const int64_t *slices_i,
                           const int64_t *redranges_j, int64_t nrj, float *out, void *stream);
int keops_gauss_lse_ranges(const float *x, const float *y, const float *b, int64_t M, int64_t N, int32_t D,
                           int32_t E, float sigma, const int64_t *ranges_i, int64_t nri, const int64_t *slices_i,
                           const int64_t *redranges_j, int64_t nrj, float *out, void *stream);
int keops_gauss_grad_x_ranges(const float *x, const float *y, const float *b, const float *g, int64_t M, int64_t N,
                              int32_t D, int32_t E, float sigma, const int64_t *ranges_i, int64_t nri,
                              const int64_t *slices_i, const int64_t *redranges_j, int64_t nrj, float *out,
                              void *stream);

/*
 * Conjugate-gradient solve of (K + lambda I) a = b with the Gaussian kernel
 * matrix of one point set, K_ij = exp(-|x_i - x_j|^2/sigma^2) ([README] feature
 * list: a conjugate gradient solver for spline interpolation, kriging or
 * Gaussian process regression).  Each of the E <= 4 columns of b is solved
 * independently, starting from a = 0, until |r_e| <= rtol |b_e| for every
 * column (r the recursively updated residual) or after max_iter iterations.
 * Every product K p is one keops_gauss_sum.
 *   x: [N, D]; b, out (= a): [N, E]; sigma > 0; lambda >= 0; rtol >= 0.
 *   iters (host, may be NULL): iterations run.
 *   rel_residual (host [E], may be NULL): the true |b - (K + lambda I) a| / |b|
 *     of the returned a, from one more product (0 for a zero column of b).
 * Unlike the reductions above this call synchronises `stream`: it reads the
 * residual norms on the host after every iteration.  Returns KEOPS_OK also when
 * max_iter is reached first (see iters and rel_residual); N = 0 is a no-op.
 */
int keops_gauss_cg(const float *x, const float *b, int64_t N, int32_t D, int32_t E, float sigma, float lambda,
                   float rtol, int32_t max_iter, float *out, int32_t *iters, float *rel_residual, void *stream);

/*
 * K-min reduction with indices ([KO-GPU] §2 argmin / argKmin; [README] ArgMin,
 * K-min reductions): for each row i, the K smallest squared distances
 * |x_i - y_j|^2, ascending, and their indices j; equal distances are ordered
 * by smaller j first.  K = 1 is ArgMin.
 * The argument list follows the other reductions, (x, y, b, ..., sigma, out,
 * stream): b and sigma do not enter a nearest-neighbour search, are never read
 * and are not validated (b may be NULL, sigma any value).
 * out_d: [M, K] fp32; out_idx: [M, K] int64, 8-byte aligned.
 * Requires 1 <= K <= N < 2^31.
 */
int keops_kmin(const float *x, const float *y, const float *b,
               int64_t M, int64_t N, int32_t D, int32_t K, float sigma,
               float *out_d, int64_t *out_idx, void *stream);

/*
 * ---------------------------------------------------------------------------
 * Paged key/value cache and draft verification (serving large language models)
 * ---------------------------------------------------------------------------
 * Attention is the same kind of reduction as above, over keys in place of points:
 * softmax(scale <q_i, k_j>) is a LogSumExp over j, its output the sum of
 * exp(z_ij - lse_i) v_j.  The keys and values of a batch of sequences lie in a pool of
 * pages; nothing of the size queries x keys is stored, but for the scores of a step that
 * asks for attention weights (below).
 *
 * Conventions of these entry points, beside the common ones:
 *  Sequence s has lens[s] slots; its starts[s+1] - starts[s] new tokens, rows starts[s] ..
 *  of the token arrays, are its last slots.  Slot j lies in row j % page_size of page
 *  page_table[s][j / page_size].  A slot whose table entry is outside [0, pages), or past
 *  the table's width, is absent: attention does not see it, append, weights and eviction
 *  leave it out.
 *  lens, starts, tables and scales are device arrays (int32, fp32).  They are read by the
 *  kernels only: a sequence with more new tokens than max_q or more slots than max_len is
 *  cut to them, starts outside [0, tokens] likewise; outputs of tokens in no sequence, or
 *  past max_q, are undefined.
 *  Strides count elements; the last dimension of every array is contiguous.  k_pages,
 *  v_pages, q, k, v and out are 16-byte aligned, their strides multiples of 16 bytes.
 *  A page in the tables of several sequences is read for each; it holds the weights of one of them.
 *  At most 2^30 slots a sequence.  Work of 2^32 threads or more in one launch (some 68 GB of
 *  keys to append or to move in 16-byte pieces) is KEOPS_ERR_UNSUPPORTED.
 *  k_pages and v_pages share their strides: [pages][page_size][heads][dim] in any order of
 *  the first three.  dim: 64, 96, 128 or 256.
 *  Types: KEOPS_TYPE_BF16 or _F16 for q, k, v, out, with a cache of the same type, of
 *  KEOPS_TYPE_E4M3 (OCP e4m3, finite to 448), whose elements stand for value * scale[head],
 *  or of KEOPS_TYPE_E2M1: 4 bits an element (OCP e2m1: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign),
 *  two to a byte, the first in its low half; each 32 columns of a row share a power of two, a
 *  byte b that stands for 2^(b - 127), 255 for NaN.  The powers of keys and values are dense
 *  arrays [pages][heads][page_size][dim / 32], 16-byte aligned, of at most 2^32 - 1 slots and
 *  heads.  A held value is read as the nearest one of the rows' type (bf16: exact but for
 *  powers past 252, fp16: exact for powers of 104 to 140).
 *  KEOPS_TYPE_F32 is for keops_rotary and keops_adjust_logits only.
 */
#define KEOPS_TYPE_BF16 0
#define KEOPS_TYPE_F16 1
#define KEOPS_TYPE_E4M3 2
#define KEOPS_TYPE_F32 3
#define KEOPS_TYPE_E2M1 4

typedef struct {
  void *k_pages, *v_pages;
  float *weights;                 /* [pages][heads][page_size], or NULL          */
  union {
    const float *k_scale;         /* [heads]; KEOPS_TYPE_E4M3 only (eviction does not read them) */
    uint8_t *k_powers;            /* KEOPS_TYPE_E2M1: of the blocks                */
  };
  union {
    const float *v_scale;
    uint8_t *v_powers;
  };
  int64_t page_stride, slot_stride, head_stride;
  int64_t pages;
  const int32_t *page_table;      /* [seqs][table_width], rows table_stride apart */
  int64_t table_stride;
  const int32_t *lens;            /* [seqs]                                      */
  int32_t page_size, heads, dim, type, table_width, seqs;
} keops_cache_t;

/*
 * New keys and values into their slots: row t of k and v ([tokens][heads][dim], rows
 * k_stride and v_stride apart) to the slot of token t.  E4M3 caches hold the value nearest
 * to k / k_scale[head] (ties to even), cut to +-448; NaN stays NaN.  Where the cache has
 * weights, those of the written slots become 0.  starts: [seqs + 1].
 * E2M1 caches: a block of 32 columns takes the least power under which none of them rounds to
 * more than 6 (at most 2^125 for bf16 rows and 2^13 for fp16 ones, so that held values are
 * finite in the rows' type; elements past 6 under that are cut to it), each column the nearest
 * value, halfway the one with the even code.  A block with a NaN or an infinity becomes NaN.
 */
int keops_cache_append(const keops_cache_t *cache, const void *k, const void *v, int64_t k_stride, int64_t v_stride,
                       int32_t type, const int32_t *starts, int64_t tokens, void *stream);

/*
 * Rotary positions.  Pair i of a head turns by the angle position * freqs[i] (64 bits, the
 * product as it is; angles up to 2^50):
 *   a' = factor (a cos - b sin),  b' = factor (a sin + b cos)
 * Half layout: a is column i, b column i + pairs; interleaved: columns 2 i and 2 i + 1.
 * Columns from 2 pairs on stay as they are.  Scaled frequencies and a factor other than 1 serve
 * texts longer than those that a model was trained on.
 */
typedef struct {
  const double *freqs;            /* [pairs], radians a position; device           */
  double factor;
  int32_t pairs;                  /* 2 pairs <= dim                                */
  int32_t interleaved;
} keops_rotary_t;

/*
 * out = x rotated, x [tokens][heads][dim] of KEOPS_TYPE_BF16, _F16 or _F32, token t's row at
 * x + t x_stride, its heads dense; out likewise, out_stride at least a row.  dim up to 65536,
 * pairs up to 8192, element-aligned; heads of whole aligned 16 bytes run fastest.  out may be x
 * itself, with the same stride, and must not overlap it otherwise.
 * inverse: the angles' signs turned, which with the same factor is the gradient: out = dL/dx for
 * x = dL/dout.  positions: [tokens] int32, of either sign.
 */
int keops_rotary(const void *x, int64_t x_stride, int32_t type, int64_t tokens, int32_t heads, int32_t dim,
                 const int32_t *positions, const keops_rotary_t *rotary, int32_t inverse, void *out, int64_t out_stride,
                 void *stream);

/*
 * keops_cache_append with rotary positions on the way: q_out = q rotated, k rotated into its
 * slot, v into its slot as it is.  The position of token t is positions[t], or, where positions
 * is NULL, the number of its slot.  Rounded once: an 8-bit or 4-bit cache holds what is nearest
 * to the rotated key (E4M3: its quotient) itself.  q: [tokens][heads][dim], rows q_stride apart;
 * q_out likewise, q_out_stride apart, heads any number (0: no q, q_out is not read); it must not
 * overlap q (a token's pieces are read by several threads), k, v or the pool.  Rows of q_out
 * of tokens in no sequence stay as they were; a token without a slot has its q rotated.
 */
int keops_cache_append_rotary(const keops_cache_t *cache, const void *q, const void *k, const void *v, int64_t q_stride,
                              int64_t k_stride, int64_t v_stride, int32_t type, int32_t heads, const int32_t *starts,
                              int64_t tokens, const int32_t *positions, const keops_rotary_t *rotary, void *q_out,
                              int64_t q_out_stride, void *stream);

/*
 * The values held in the slots of every sequence's last starts[s+1] - starts[s] tokens, as 16-bit
 * rows: k and v [tokens][heads][dim], rows k_stride and v_stride apart (starts 0 .. lens: whole
 * sequences).  type: the cache's own, or either 16-bit one of an 8-bit or 4-bit cache, to nearest.
 * Rows of slots that are absent are 0, those of tokens in no sequence stay as they were.
 */
int keops_cache_read(const keops_cache_t *cache, void *k, void *v, int64_t k_stride, int64_t v_stride, int32_t type,
                     const int32_t *starts, int64_t tokens, void *stream);

/*
 * Causal attention of every sequence's new tokens over its slots:
 *   z_j = scale <q[t, g], k_j>,  lse[t, g] = log sum_j exp(z_j),  out[t, g] = sum_j exp(z_j - lse) v_j
 * over the slots j <= the token's own, and, with window > 0, j > its own - window.  heads
 * query heads, a multiple of the cache's; query head g reads key/value head
 * g / (heads / cache heads).  A token that sees no slot has out = 0 and lse = -inf.
 * q: [tokens][heads][dim], rows q_stride apart; out: the same shape, dense; lse: [tokens][heads].
 * Where the cache has weights, slot j's becomes
 *   decay * old + sum over the new tokens t and the query heads g of the key/value head of exp(z_j - lse)
 * for every slot of every sequence (decay = 0 does not read the old ones; 1 accumulates), also
 * where no sequence has a new token.
 * A value that a row does not see has no effect on it, whatever it holds.
 * workspace: NULL for the library's (see "Ownership" above), or a 256-byte aligned device
 * buffer of at least keops_paged_attention_workspace bytes (KEOPS_ERR_SCRATCH if smaller).
 * Under stream capture a call that needs workspace must bring its own (KEOPS_ERR_ALLOC
 * otherwise), which has to live as long as the graph.  Prompts over an E2M1 cache take up to 4 GB
 * to hold its slots in 16 bits; where the library cannot allocate that, they do without: the same
 * bits, slower.
 */
int keops_paged_attention(const keops_cache_t *cache, const void *q, int64_t q_stride, int32_t type, int32_t heads,
                          const int32_t *starts, int64_t tokens, int32_t max_q, int32_t max_len, float scale,
                          int32_t window, float decay, void *out, float *lse, void *workspace, int64_t workspace_bytes,
                          void *stream);

/* Workspace bytes of a keops_paged_attention call with these arguments on the current device. */
int keops_paged_attention_workspace(const keops_cache_t *cache, int32_t type, int32_t heads, int64_t tokens,
                                    int32_t max_q, int32_t max_len, int32_t window, int64_t *bytes);

/*
 * Eviction by attention weight.  Of a sequence's slots that are not absent each key/value
 * head keeps `budget`: those among the first `sink` slots, those among the last `recent`, and
 * of the others the ones with the largest weights (equal weights: the lower slot; NaN is
 * largest); where there are no more than `budget`, all.  Absent slots are left out, so a table
 * with holes ends without them.  Kept slots move in their
 * order to slots 0 .. of the pages of new_table ([seqs][new_width], rows new_stride apart):
 * keys, values and weights.  Pages of new_table are none of page_table's, and no page is in
 * new_table twice (their contents are undefined otherwise).
 * kept: [seqs][heads][budget], the old slot numbers, -1 past the end; new_lens: [seqs], the
 * smaller of `budget` and the slots that are not absent.
 * new_width >= min(ceil(budget / page_size), table_width); 1 <= budget, sink + recent <= budget.
 */
int keops_cache_evict(const keops_cache_t *cache, const int32_t *new_table, int64_t new_stride, int32_t new_width,
                      int32_t budget, int32_t sink, int32_t recent, int32_t *kept, int32_t *new_lens, void *stream);

/*
 * Verification of drafted tokens.  Sequence s drafted tokens[s][0 .. counts[s]) from
 * draft[s][r][.]; target[s][r][.] are the target model's probabilities at the same places
 * and at the one after (fp32, each row's scale free).  Token r is taken while
 *   u_accept[s][r] * draft[s][r][x] < target[s][r][x];
 * the token after the taken ones is the lowest index whose running sum of the mass m
 * exceeds u_sample[s] times the total, with m = max(target - draft, 0) at a refused place
 * (target itself if that is 0 everywhere) and m = target after the last.  Sums in 64 bits.
 * draft = NULL: the drafted token had probability 1.  A token outside [0, vocab) is refused.
 * target: [seqs][drafts + 1][vocab], draft: [seqs][drafts][vocab], tokens, u_accept:
 * [seqs][drafts]; out: [seqs][drafts + 1], the taken tokens, the new one, then -1;
 * accepted: [seqs], how many were taken.  workspace: as for keops_paged_attention.
 */
int keops_verify_draft(const float *target, const float *draft, const int32_t *tokens, const int32_t *counts,
                       const float *u_accept, const float *u_sample, int32_t seqs, int32_t drafts, int32_t vocab,
                       int32_t *out, int32_t *accepted, void *workspace, int64_t workspace_bytes, void *stream);

/* Workspace bytes of a keops_verify_draft call. */
int keops_verify_draft_workspace(int32_t seqs, int32_t drafts, int32_t vocab, int64_t *bytes);

/*
 * Logits by a text's penalties, biases and masks.  Row r of sequence s (rows starts[s] ..
 * starts[s+1]) has seen the text up to token j = lens[s] - (starts[s+1] - starts[s]) + r, as a
 * token's query has seen the slots up to its own; a row before the text's start has seen nothing.
 * With c the times that a vocabulary entry x occurs among text[s][prompt_lens[s] .. j]:
 *   z = logits[t][x]
 *   if x occurs in text[s][0 .. j]:  z = z > 0 ? z / repetition[s] : z * repetition[s]
 *   z = z - frequency[s] c - (c > 0 ? presence[s] : 0) + (bias of x in the list of s, if any)
 *   z = -inf where x's bit of the row's mask is 0
 * in 64 bits where a rule touches an entry, rounded once; untouched entries stay as they are.
 * A NULL array leaves its rule out.  Entries of text and bias_tokens outside [0, vocab) count for
 * nothing; of several equal bias_tokens the last stands.  mask: [rows][ceil(vocab / 32)], bit
 * x % 32 of word x / 32, rows mask_stride apart.  Rows of no sequence stay as they were.
 * logits and out: [rows][vocab] of KEOPS_TYPE_BF16, _F16 or _F32, rows stride and out_stride
 * apart; out may be logits itself, with the same stride, and must not overlap it otherwise.
 * vocab and biases up to 2^30, text_width below that.
 */
typedef struct {
  const int32_t *starts;          /* [seqs + 1]                                    */
  const int32_t *text;            /* [seqs][text_width], rows text_stride apart    */
  int64_t text_stride;
  const int32_t *lens;            /* [seqs], needed with text                      */
  const int32_t *prompt_lens;     /* [seqs]; NULL: 0                               */
  const float *repetition, *presence, *frequency;     /* [seqs], with text         */
  const int32_t *bias_tokens;     /* [seqs][biases], dense                         */
  const float *bias;              /* [seqs][biases]                                */
  const int32_t *mask;
  int64_t mask_stride;
  int32_t seqs, text_width, biases;
} keops_logit_rules_t;

int keops_adjust_logits(const void *logits, int64_t stride, int32_t type, int64_t rows, int32_t vocab,
                        const keops_logit_rules_t *rules, void *out, int64_t out_stride, void *stream);

/* Human-readable name of a status code (static storage). */
const char *keops_status_string(int status);

/*
 * Process-wide tuning and test switches (0 = automatic for each).  They change
 * how the work is scheduled, never what is computed beyond fp32 rounding:
 *   KEOPS_OPT_SPLIT_J   -- force this many j-splits (pass 1 partials + pass 2)
 *   KEOPS_OPT_FORM      -- 1 = use the direct distance form everywhere (the
 *                          expanded form is otherwise used wherever its range
 *                          condition holds)
 *   KEOPS_OPT_ROWS      -- 1 = one row per lane, 2 = the wide variant (several
 *                          rows per lane, for large M), 3 = the few-rows layout
 *                          of the sum, LogSumExp, gradient with respect to x
 *                          and K-min (j per lane, rows in LDS or registers;
 *                          chosen automatically for M <= 64 at D <= 8)
 *   KEOPS_OPT_WG_TARGET -- work-groups per CU the automatic j-split aims for
 *                          (1..4096; ignored when KEOPS_OPT_SPLIT_J is set)
 *   KEOPS_OPT_MFMA      -- 1 = the Gaussian sum and K-min never use the
 *                          matrix cores (the VALU expanded form runs at every
 *                          D; automatically they are used for D >= 32);
 *                          2 = the K-min prefilter at D >= 32 takes the fp32
 *                          MFMA form instead of the split-bf16 one (the same
 *                          results; the sum is unaffected)
 *   KEOPS_OPT_WS_CACHE  -- 2 = no workspace cache: every call allocates and
 *                          frees its workspace in stream order
 *                          (hipMallocAsync / hipFreeAsync); setting it also
 *                          frees the cached buffers no call holds
 *   KEOPS_OPT_FAIL_ALLOC -- test switch: 1 = every workspace allocation fails,
 *                          so that a call needing workspace returns
 *                          KEOPS_ERR_ALLOC with nothing enqueued (or takes a
 *                          form without workspace, if it has one)
 * Returns KEOPS_OK, or KEOPS_ERR_INVALID_ARG for an unknown option or value.
 */
#define KEOPS_OPT_SPLIT_J 1
#define KEOPS_OPT_FORM 2
#define KEOPS_OPT_ROWS 3
#define KEOPS_OPT_PROFILE 4   /* 1 = record HIP events around each pass-1 launch */
#define KEOPS_OPT_WG_TARGET 5
#define KEOPS_OPT_MFMA 6
#define KEOPS_OPT_WS_CACHE 7
#define KEOPS_OPT_FAIL_ALLOC 8
int keops_set_option(int option, int64_t value);

/*
 * Duration of the pass-1 (pair-evaluation) kernels, for benchmarks.  While
 * KEOPS_OPT_PROFILE is 1, every call records a HIP event pair around its
 * pass-1 launch on the call's stream (at most 4096 pairs are kept).  This
 * waits for the recorded events, returns the summed duration in milliseconds
 * and the number of launches since the previous read, and forgets them.
 * total_ms and launches must be valid host pointers.
 */
int keops_profile_read(double *total_ms, int64_t *launches);

/* Library version as 10000*major + 100*minor + patch. */
int keops_version(void);

#ifdef __cplusplus
}
#endif

#endif /* KEOPS_MI355X_H */
