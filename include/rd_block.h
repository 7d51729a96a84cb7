/*
 * rd_block.h -- C ABI of the rest of a feed-forward block around the experts: the norm in front of
 * the router and the products, products with a bias, an activation and a residual (the router's
 * logits, experts with biases, a dense or shared feed-forward beside them), and dropout with the
 * residual behind.
 *
 * The rules of rd.h hold here too: plain device pointers and sizes, work enqueued on the caller's
 * stream, no synchronisation, no allocation, no copy to the host, capturable in a CUDA graph;
 * the caller owns every buffer, workspaces included (two graphs that may replay at the same time
 * need a workspace each); invalid arguments are rejected before anything is enqueued.
 * Matrices are row-major and contiguous.  The first call of each entry point in a process sets
 * kernel attributes; make it before a stream capture begins.
 *
 * Types: `dtype` and `out_dtype` are RD_F32 or RD_BF16 (rd_moe.h) and independent of one another;
 * everything in between is f32, with one rounding at the end.  Matrices start on 16-byte
 * boundaries, f32 matrices on 32-byte ones, vectors of f32 (weight, bias, their gradients) on
 * 16-byte ones, row statistics on 4-byte ones.  Outputs overlap nothing.
 *
 * Where a call takes `limit` (device int32 or NULL), L = min(max(*limit, 0), rows): rows at or past L
 * are neither read nor written and enter no sum.
 */
#ifndef RD_BLOCK_H_
#define RD_BLOCK_H_

#include "rd_moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * rd_layer_norm_fwd -- out[r, c] = (x[r, c] - mean[r]) * rstd[r] * weight[c] + bias[c]
 *   mean[r] = sum_c x[r, c] / hidden,  rstd[r] = 1 / sqrt(sum_c (x[r, c] - mean[r])^2 / hidden + eps)
 *   The squares are summed about the mean, so rows far from zero keep their variance.
 *   x [rows, hidden] of `dtype`, out [rows, hidden] of `out_dtype`; weight, bias [hidden] f32, NULL
 *   for ones and zeros; mean, rstd [rows] f32: both (the backward pass reads them) or both NULL.
 * Requires hidden % 8 == 0, eps finite and >= 0 (with eps = 0 a constant row gives NaN).
 */
rd_status rd_layer_norm_fwd(const void* x, int32_t dtype, const float* weight, const float* bias,
                            float eps, void* out, int32_t out_dtype, float* mean, float* rstd,
                            int64_t rows, int64_t hidden, const int32_t* limit, rd_stream_t stream);

/*
 * rd_layer_norm_bwd -- the gradients of rd_layer_norm_fwd.  With y = (x - mean) * rstd, g = d_out * weight:
 *   d_x[r, c]   = rstd[r] * (g[r, c] - sum_j g[r, j] / hidden - y[r, c] * sum_j g[r, j] y[r, j] / hidden)
 *   d_weight[c] = sum_{r < L} d_out[r, c] * y[r, c]      (f32)
 *   d_bias[c]   = sum_{r < L} d_out[r, c]                (f32)
 *   d_out of `out_dtype`, x and d_x of `dtype`, weight [hidden] f32 or NULL, mean, rstd [rows] f32.
 *   d_weight, d_bias [hidden] f32, either NULL to leave it out.  No atomics: the same result on every run.
 *   workspace  device scratch of rd_layer_norm_bwd_workspace_size bytes, 32-byte aligned; may be
 *              NULL when both d_weight and d_bias are, or that size is 0.  Its contents before and
 *              after do not matter.
 * Rows of 8200 to 65536 elements are shared by blocks that wait for one another's sums, each wait bounded as those of rd.h are
 * (rd_set_tuning's wait_timeout_ns).  There is no status word: where a wait runs out, d_x is NaN from the row it was for
 * on, in that block's columns of the rows that it takes, and soon in those of the blocks that share them; every other
 * element of d_x, d_weight and d_bias is what it would be otherwise.
 * Requires hidden % 8 == 0.
 */
rd_status rd_layer_norm_bwd(const void* d_out, int32_t out_dtype, const void* x, int32_t dtype,
                            const float* weight, const float* mean, const float* rstd, void* d_x,
                            float* d_weight, float* d_bias, int64_t rows, int64_t hidden,
                            const int32_t* limit, void* workspace, size_t workspace_bytes,
                            rd_stream_t stream);

/* The workspace of rd_layer_norm_bwd on the current device; 0 where it needs none (few rows). */
rd_status rd_layer_norm_bwd_workspace_size(int64_t rows, int64_t hidden, size_t* bytes);

/* activations of rd_linear */
#define RD_ACT_NONE 0
#define RD_ACT_RELU 1
#define RD_ACT_GELU 2      /* z * P(z), P the normal distribution function */
#define RD_ACT_GELU_TANH 3 /* z / 2 * (1 + tanh(sqrt(2 / pi) * (z + 0.044715 z^3))) */
#define RD_ACT_SILU 4      /* z / (1 + exp(-z)) */

/*
 * rd_linear -- rows times weights with bias, activation and residual in the product's epilogue.
 *   z[i, :]   = x[i, :] @ w[j, :, :] + bias[j, :]   (f32)    for every row i of local group j
 *   pre[i, :] = bf16(z[i, :])                                where pre is not NULL
 *   out[i, :] = act(z[i, :]) + residual[i, :]
 *   group_sizes NULL: one weight for all rows, w [k, n], bias [n] (g_total = g_local = 1, group_offset = 0).
 *   Otherwise groups, group_offset, limit and status as rd_ragged_dot, w [g_local, k, n], bias
 *   [g_local, n]; rows in [0, L) outside the local groups are +0 in out and pre (no residual).
 *   x [m, k], w, pre [m, n] bf16; bias f32 or NULL; out and residual (or NULL) [m, n] of `out_dtype`.
 * Accuracy: the products are exact and summed in f32 by the tensor cores, which cut the sum off at every 16 of k;
 * an f32 output adds up stretches of 512 of k with rounding (some 5e-7 of the output's norm, whatever k is).
 * Activations are within 4e-6 + 5e-7 |u| of their value, relatively, u the argument of their exponential (z^2 / 2,
 * 2 sqrt(2 / pi) (z + 0.044715 z^3) or z); silu's values below 1.1e-36 and gelu's, in both forms, below 1.2e-37 may be 0.
 * Its gradients: rd_linear_act_bwd gives d_pre and d_bias; dx is rd_ragged_dot_trans_rhs(d_pre, w),
 * dw is rd_trans_ragged_dot(x, d_pre) (one weight: with group_sizes a word that holds m), and the
 * residual's gradient is d_out.
 * Requires k % 8 == 0, n % 8 == 0, n at most 2^31 - 256.
 */
rd_status rd_linear(const void* x, const void* w, const float* bias, const void* residual,
                    int32_t act, void* out, int32_t out_dtype, void* pre, int64_t m, int64_t k,
                    int64_t n, const int32_t* group_sizes, int32_t g_total, int32_t group_offset,
                    int32_t g_local, const int32_t* limit, int32_t* status, rd_stream_t stream);

/*
 * rd_linear_act_bwd -- gradients of rd_linear in front of its activation, in one pass.
 *   d_z[i, c]    = d_out[i, c] * act'(pre[i, c])    (f32; relu has slope 0 at 0)
 *   d_pre[i, c]  = bf16(d_z[i, c])                  where d_pre is not NULL
 *   d_bias[j, c] = sum of d_z[i, c] over the rows i of local group j    (f32, of the unrounded d_z),
 *                  where d_bias is not NULL; a group without rows gives 0
 *   Groups as rd_linear: rows of d_pre in [0, L) outside the local groups are +0.
 *   d_out [m, n] of `out_dtype`, pre [m, n] bf16 (NULL with RD_ACT_NONE), d_pre [m, n] bf16, d_bias [g_local, n].
 *   act'(z) = P + z P' for the activation z P(z); it is within 4e-6 + 5e-7 |u| (as for rd_linear) of |P| + |z P'|, relatively,
 *   and 0 may stand for what is below 3e-36.
 *   No atomics: the same result on every run.
 *   workspace  device scratch of rd_linear_act_bwd_workspace_size bytes, 32-byte aligned; may be NULL
 *              when d_bias is or that size is 0.  Its contents before and after do not matter.
 * Requires n % 8 == 0.
 */
rd_status rd_linear_act_bwd(const void* d_out, int32_t out_dtype, const void* pre, int32_t act,
                            void* d_pre, float* d_bias, int64_t m, int64_t n,
                            const int32_t* group_sizes, int32_t g_total, int32_t group_offset,
                            int32_t g_local, const int32_t* limit, void* workspace,
                            size_t workspace_bytes, int32_t* status, rd_stream_t stream);

/* The workspace of rd_linear_act_bwd; 0 where it needs none (few rows). */
rd_status rd_linear_act_bwd_workspace_size(int64_t m, int64_t n, int32_t g_local, size_t* bytes);

/*
 * rd_dropout_rows -- out = kept(x) * scale + residual, by a counter-based generator; no mask is stored.
 *   Elements (r, c) come in vectors of eight, vector v = (r * hidden + c) / 8.  The generator (Philox
 *   4x32 in ten rounds: J. Salmon et al., "Parallel random numbers: as easy as 1, 2, 3", 2011) gives
 *   four 32-bit words for the key (low, high word of rng[0]) and the counter (low, high word of v, low, high
 *   word of rng[1]); element i of the vector has the 16 bits i % 2 (0: the low ones) of word i / 2.
 *   It is kept where they are >= T = round(65536 p), halves up; scale = 65536 / (65536 - T), so the mean is x for
 *   the p that is used, a multiple of 2^-16.  p = 1 keeps nothing.  A dropped element is 0 whatever
 *   its value.
 *   rng [2] int64 (a seed and an offset) is read on the device: a captured graph draws anew when the
 *   words change between replays.
 *   x [rows, hidden] of `dtype`, residual (or NULL) and out [rows, hidden] of `out_dtype`.
 * The gradient of x is the same call on the gradient of out, with the same rng and p, without
 * residual; that of the residual is the gradient of out.
 * Requires hidden % 8 == 0, 0 <= p <= 1, rng 8-byte aligned.
 */
rd_status rd_dropout_rows(const void* x, int32_t dtype, const void* residual, const int64_t* rng,
                          float p, void* out, int32_t out_dtype, int64_t rows, int64_t hidden,
                          const int32_t* limit, rd_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* RD_BLOCK_H_ */
