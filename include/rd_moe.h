/*
 * rd_moe.h -- C ABI of the operators around the grouped expert products of rd.h: routing tokens
 * to experts, sorting them into the packed buffer and back, and the experts' products in 4 bits.
 *
 * The rules of rd.h hold here too: plain device pointers and sizes, work enqueued on the caller's
 * stream, no synchronisation, no allocation, no copy to the host, capturable in a CUDA graph;
 * the caller owns every buffer; invalid arguments are rejected before anything is enqueued.
 * Matrices are row-major and contiguous.  The first call of each entry point in a process sets
 * kernel attributes; make it before a stream capture begins.
 *
 * Tokens and packed rows.  A layer sends each of T tokens to `topk` experts; slot (t, k) is
 * token t's k-th choice.  pos[t, k] is the row of slot (t, k) in the packed buffer, whose rows are
 * sorted by expert (then by slot), so that rows of expert j are a group of rd_ragged_dot and
 * `group_sizes` its sizes.  A slot without an expert (id outside [0, experts)) has pos -1 and no
 * row.  `rows` (device) is the number of packed rows, usable as the `limit` of the grouped calls.
 *
 * Where a call takes `limit` (device int32 or NULL), L = min(max(*limit, 0), tokens): tokens at or
 * past L are neither read nor written and have no packed row.
 */
#ifndef RD_MOE_H_
#define RD_MOE_H_

#include "rd.h"

#ifdef __cplusplus
extern "C" {
#endif

/* element type of the router's logits and their gradient */
#define RD_F32 0
#define RD_BF16 1

/* scores of the router */
#define RD_SCORE_SOFTMAX 0
#define RD_SCORE_SIGMOID 1

#define RD_MAX_TOPK 32
#define RD_MAX_EXPERT_GROUPS 32

typedef struct {
  int32_t topk;         /* experts per token, 1 .. min(experts, RD_MAX_TOPK) */
  int32_t score;        /* RD_SCORE_SOFTMAX or RD_SCORE_SIGMOID */
  int32_t groups;       /* expert groups of equal size, 1 .. RD_MAX_EXPERT_GROUPS; divides experts */
  int32_t topk_groups;  /* groups a token may use, 1 .. groups */
  int32_t renormalize;  /* 0: weights are the scores; 1: divided by their sum over the slots */
  float scale;          /* factor of every weight */
} rd_route_config;

/*
 * rd_route -- scores, choice of experts and weights; optionally the plan of the packed buffer.
 *   A logit l of -inf or NaN masks its expert for that token: it is never chosen.
 *   softmax: key = l + bias;                     group score = the group's largest key
 *   sigmoid: s = 1 / (1 + exp(-l)), key = s + bias; group score = the sum of the group's two
 *            largest keys (a missing second one counts as 0)
 *   The topk_groups best groups are kept (all of them when groups = 1) and the topk best experts
 *   among them chosen, best first; ties go to the lower index (zeros of either sign tie).  A group
 *   without an unmasked expert is never kept.  Slots left without an expert get id -1 and weight 0.
 *   weights (f32): softmax  scale * exp(l - max) / sum over all unmasked experts, or, renormalised,
 *                  scale * the softmax over the chosen logits (the bias does not enter);
 *                  sigmoid  scale * s, or, renormalised, scale * s / (sum of the chosen s),
 *                  which is 0 where that sum is 0.
 *   All in f32, with the accurate exp and division, so that the keys, and with them the ids,
 *   equal those of the same formulas in elementwise f32 arithmetic (where exp(-l) overflows, at
 *   l < -88.7, the sigmoid is 0).  A logit of +inf gives NaN softmax weights.
 *
 *   logits  [tokens, experts] f32 or bf16 (`dtype`), experts 1 .. RD_MAX_GROUPS
 *   bias    [experts] f32 or NULL (a load-balancing term: it moves the choice, not the weights)
 *   ids     [tokens, topk] int32,  weights [tokens, topk] f32
 *   group_sizes [experts], pos [tokens, topk], rows [1] int32: the plan of rd_sort_rows, or all
 *           three NULL to leave it out
 * No alignment beyond the element type's.
 */
rd_status rd_route(const void* logits, int32_t dtype, const float* bias, int64_t tokens,
                   int64_t experts, const rd_route_config* config, const int32_t* limit,
                   int32_t* ids, float* weights, int32_t* group_sizes, int32_t* pos, int32_t* rows,
                   rd_stream_t stream);

/*
 * rd_route_bwd -- gradient of the logits from the gradient of the weights.
 *   With q the weights divided by scale, S the sum that renormalisation divides by, d the given
 *   gradients and the sums over the slots of the token that have an expert:
 *   softmax                 d_l[j] = scale * p_j * ((j chosen) * d_j - sum_k q_k d_k), every expert
 *   softmax, renormalised   d_l[j] = scale * q_j * (d_j - sum_k q_k d_k) on the chosen ones
 *   sigmoid                 d_l[j] = scale * d_j * s_j * (1 - s_j) on the chosen ones
 *   sigmoid, renormalised   d_l[j] = scale / S * (d_j - sum_k q_k d_k) * s_j * (1 - s_j), chosen
 *   and 0 elsewhere (masked experts included); the choice itself has no gradient.  Computed in
 *   f32, rounded once.  An id outside [0, experts) is a slot without an expert; the ids of one
 *   token must differ.
 *
 *   logits, d_logits [tokens, experts] of type `dtype`, ids [tokens, topk] int32,
 *   d_weights [tokens, topk] f32.  Of config, groups and topk_groups are not used.
 */
rd_status rd_route_bwd(const void* logits, int32_t dtype, const int32_t* ids,
                       const float* d_weights, int64_t tokens, int64_t experts,
                       const rd_route_config* config, const int32_t* limit, void* d_logits,
                       rd_stream_t stream);

/*
 * rd_sort_rows -- the plan of the packed buffer from the slots' expert ids (a stable counting
 * sort: by expert, then by slot; the same on every run).
 *   ids [tokens, topk] int32 -> group_sizes [experts], pos [tokens, topk], rows [1], int32.
 */
rd_status rd_sort_rows(const int32_t* ids, int64_t tokens, int64_t topk, int64_t experts,
                       const int32_t* limit, int32_t* group_sizes, int32_t* pos, int32_t* rows,
                       rd_stream_t stream);

/*
 * rd_dispatch_rows -- out[pos[t, k], :] = x[t, :] for every slot with a row.  x is read once.
 *   x [tokens, hidden] bf16, pos [tokens, topk] int32, out [out_rows, hidden] bf16.  A position
 *   outside [0, out_rows) is skipped; rows of out that no slot has stay as they are.
 * The gradient of x is rd_combine_rows of the gradient of out, without weights.
 * Requires hidden % 8 == 0, 16-byte aligned matrices, no overlap.
 */
rd_status rd_dispatch_rows(const void* x, const int32_t* pos, void* out, int64_t tokens,
                           int64_t topk, int64_t hidden, int64_t out_rows, const int32_t* limit,
                           rd_stream_t stream);

/*
 * rd_combine_rows -- out[t, :] = bf16(sum_k w[t, k] * y[pos[t, k], :]), summed in f32 in the order
 * of k.  A slot whose position is outside [0, y_rows) adds nothing (whatever its weight).
 *   y [y_rows, hidden] bf16, pos [tokens, topk] int32, w [tokens, topk] f32 or NULL (ones),
 *   out [tokens, hidden] bf16.
 * Requires hidden % 8 == 0, 16-byte aligned matrices, no overlap.
 */
rd_status rd_combine_rows(const void* y, const int32_t* pos, const float* w, void* out,
                          int64_t tokens, int64_t topk, int64_t hidden, int64_t y_rows,
                          const int32_t* limit, rd_stream_t stream);

/*
 * rd_combine_rows_bwd -- both gradients of rd_combine_rows in one pass.
 *   d_y[pos[t, k], :] = bf16(w[t, k] * d_out[t, :])
 *   d_w[t, k]         = sum_c d_out[t, c] * y[pos[t, k], c]   (f32; 0 for a slot without a row)
 *   Rows of d_y that no slot has stay as they are.  Each sum belongs to one warp: no atomics, the
 *   same result on every run.
 */
rd_status rd_combine_rows_bwd(const void* d_out, const void* y, const int32_t* pos, const float* w,
                              void* d_y, float* d_w, int64_t tokens, int64_t topk, int64_t hidden,
                              int64_t y_rows, const int32_t* limit, rd_stream_t stream);

/*
 * Microscaled 4-bit rows (OCP Microscaling MXFP4).  A row of k elements (k % 32 == 0) is held as
 *   q      k / 2 bytes: E2M1 codes (sign, magnitudes 0 0.5 1 1.5 2 3 4 6), element 2i in the low
 *          half of byte i
 *   scales rd_mxfp4_scale_width(k) bytes (k / 32 rounded up to a multiple of 16): byte b is the
 *          E8M0 scale 2^(scales[b] - 127) of elements [32 b, 32 b + 32), 0xFF stands for NaN; the
 *          bytes from k / 32 on are not read
 * Quantisation of a block: e = floor(log2(largest magnitude)) - 2, at least -127; code = x / 2^e
 * rounded to nearest even, magnitudes above 6 to 6 (the exponent is that of the format's own
 * definition, so the largest magnitude of a block may be cut by up to a quarter).  A block with a
 * NaN or an infinity gets scale 0xFF and codes 0.
 */
int64_t rd_mxfp4_scale_width(int64_t k);

/*
 * rd_mxfp4_quantize -- bf16 rows to 4-bit rows, optionally sent to their packed rows on the way.
 *   pos NULL: row r of x becomes row r of q and scales (out_rows >= rows, topk ignored).
 *   pos [rows, topk] int32: row t becomes every row pos[t, k] in [0, out_rows) (rd_dispatch_rows
 *   and the quantisation in one pass over x).
 *   x [rows, k] bf16, q [out_rows, k / 2], scales [out_rows, rd_mxfp4_scale_width(k)] uint8.
 *   limit as for tokens, over the rows of x.  The scale bytes past k / 32 are written as 0.
 * Requires k % 32 == 0, 16-byte aligned matrices, no overlap.
 */
rd_status rd_mxfp4_quantize(const void* x, const int32_t* pos, void* q, void* scales, int64_t rows,
                            int64_t topk, int64_t k, int64_t out_rows, const int32_t* limit,
                            rd_stream_t stream);

/*
 * rd_mxfp4_quantize_weights -- the expert weights of rd_ragged_dot, rhs [g, k, n] bf16, to 4-bit
 * rows along k: q [g, n, k / 2], scales [g, n, rd_mxfp4_scale_width(k)].  Done once per model.
 * Requires k % 32 == 0, n % 8 == 0, 16-byte aligned matrices, no overlap.
 */
rd_status rd_mxfp4_quantize_weights(const void* rhs, void* q, void* scales, int64_t g, int64_t k,
                                    int64_t n, rd_stream_t stream);

/*
 * rd_mxfp4_dequantize -- the values of 4-bit rows as bf16: exact, except that magnitudes of 2^128 and more,
 * which scale bytes 253 and 254 (none that rd_mxfp4_quantize writes) can give, become infinities.
 *   q [rows, k / 2], scales [rows, rd_mxfp4_scale_width(k)] -> out [rows, k] bf16; rows < L only.
 */
rd_status rd_mxfp4_dequantize(const void* q, const void* scales, void* out, int64_t rows, int64_t k,
                              const int32_t* limit, rd_stream_t stream);

/* epilogues of rd_ragged_dot_mxfp4 beside RD_EPI_NONE and RD_EPI_SILU_GLU */
#define RD_EPI_SILU_GLU_MXFP4 2 /* the f32 SiLU-GLU result quantised to 4-bit rows */

/*
 * rd_ragged_dot_mxfp4 -- rd_ragged_dot over 4-bit operands, on the block-scaled tensor cores.
 *   out[i, :] = sum_k a[i, k] * b[j, :, k] for every row i of local group j; f32 accumulation.
 *   Groups, group_offset, limit, status and zero rows as rd_ragged_dot; rows of a past the groups
 *   may be read but do not enter a result.
 *   a [m, k / 2], a_scales [m, rd_mxfp4_scale_width(k)];
 *   b [g_local, n, k / 2], b_scales [g_local, n, rd_mxfp4_scale_width(k)]
 *   epi  RD_EPI_NONE      out [m, n] bf16
 *        RD_EPI_SILU_GLU  out [m, n / 2] bf16; gate = rows [0, n / 2) of b[j], up = [n / 2, n)
 *        RD_EPI_SILU_GLU_MXFP4  out [m, n / 4] bytes and out_scales [m, rd_mxfp4_scale_width(n / 2)]:
 *                         4-bit rows of width n / 2, quantised from the f32 result (the scale
 *                         bytes past n / 64 are not written); zero rows are zero bytes in both
 *   out_scales is NULL for the other two.
 * Requires k % 32 == 0, n % 8 == 0 (n / 2 % 8 == 0 with the GLU, n / 2 % 32 == 0 with the 4-bit
 * output), 16-byte aligned matrices, no overlap of the outputs with anything; k at most 2^31 - 1024 and
 * the output's width (n, n / 2 with the GLU) at most 2^31 - 256.
 */
rd_status rd_ragged_dot_mxfp4(const void* a, const void* a_scales, const void* b,
                              const void* b_scales, void* out, void* out_scales, int64_t m,
                              int64_t k, int64_t n, const int32_t* group_sizes, int32_t g_total,
                              int32_t group_offset, int32_t g_local, const int32_t* limit,
                              int32_t epi, int32_t* status, rd_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* RD_MOE_H_ */
