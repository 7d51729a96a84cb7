// api_moe.cu -- the C entry points of include/rd_moe.h: argument checks (all of those that the
// host can make come before any CUDA call), tensor maps, launch shapes.
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/rd_moe.h"
#include "gemm_mxfp4.cuh"
#include "host.h"
#include "moe_args.h"

using namespace rd;

namespace {

rd_status done(cudaError_t e) { return e == cudaSuccess ? RD_OK : RD_ERR_CUDA; }

cudaStream_t cu(rd_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

// one buffer of a call, to be checked against the others
struct Span {
  const void* p;
  uint64_t bytes;
};

// whether an output overlaps an input or another output
template <int O, int I>
bool any_overlap(const Span (&outs)[O], const Span (&ins)[I]) {
  for (int o = 0; o < O; ++o) {
    for (int i = 0; i < I; ++i)
      if (overlap(outs[o].p, outs[o].bytes, ins[i].p, ins[i].bytes)) return true;
    for (int i = 0; i < o; ++i)
      if (overlap(outs[o].p, outs[o].bytes, outs[i].p, outs[i].bytes)) return true;
  }
  return false;
}

rd_status check_route(const void* logits, int32_t dtype, int64_t tokens, int64_t experts,
                      const rd_route_config* c, const int32_t* limit) {
  if (c == nullptr || tokens < 0 || experts < 1) return RD_ERR_INVALID_ARG;
  if (dtype != RD_F32 && dtype != RD_BF16) return RD_ERR_INVALID_ARG;
  if (c->score != RD_SCORE_SOFTMAX && c->score != RD_SCORE_SIGMOID) return RD_ERR_INVALID_ARG;
  if (c->renormalize != 0 && c->renormalize != 1) return RD_ERR_INVALID_ARG;
  if (c->topk < 1 || c->topk > experts) return RD_ERR_INVALID_ARG;
  if (experts > RD_MAX_GROUPS || c->topk > RD_MAX_TOPK || tokens > kMaxDim ||
      tokens * c->topk > kMaxDim)
    return RD_ERR_UNSUPPORTED;
  if (tokens > 0 && logits == nullptr) return RD_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(logits) & (dtype == RD_F32 ? 3u : 1u)) || !aligned4(limit))
    return RD_ERR_UNSUPPORTED;
  return RD_OK;
}

RouteArgs route_args(const void* logits, const rd_route_config* c, int64_t tokens, int64_t experts,
                     const int32_t* limit) {
  RouteArgs a = {};
  a.logits = logits;
  a.limit = limit;
  a.tokens = static_cast<int32_t>(tokens);
  a.experts = static_cast<int32_t>(experts);
  a.topk = c->topk;
  a.groups = c->groups;
  a.topk_groups = c->topk_groups;
  a.score = c->score;
  a.renormalize = c->renormalize;
  a.scale = c->scale;
  return a;
}

rd_status check_sort(int64_t tokens, int64_t topk, int64_t experts, const int32_t* ids,
                     const int32_t* limit, const int32_t* group_sizes, const int32_t* pos,
                     const int32_t* rows) {
  if (tokens < 0 || topk < 1 || experts < 1) return RD_ERR_INVALID_ARG;
  if (experts > RD_MAX_GROUPS || tokens > kMaxDim || topk > kMaxDim || tokens * topk > kMaxDim)
    return RD_ERR_UNSUPPORTED;
  if (group_sizes == nullptr || rows == nullptr) return RD_ERR_INVALID_ARG;
  if (tokens > 0 && (ids == nullptr || pos == nullptr)) return RD_ERR_INVALID_ARG;
  if (!aligned4(ids) || !aligned4(limit) || !aligned4(group_sizes) || !aligned4(pos) || !aligned4(rows))
    return RD_ERR_UNSUPPORTED;
  return RD_OK;
}

}  // namespace

extern "C" rd_status rd_route(const void* logits, int32_t dtype, const float* bias, int64_t tokens,
                              int64_t experts, const rd_route_config* config, const int32_t* limit,
                              int32_t* ids, float* weights, int32_t* group_sizes, int32_t* pos,
                              int32_t* rows, rd_stream_t stream) {
  rd_status st = check_route(logits, dtype, tokens, experts, config, limit);
  if (st != RD_OK) return st;
  const int32_t groups = config->groups;
  if (groups < 1 || experts % groups != 0 || config->topk_groups < 1 || config->topk_groups > groups)
    return RD_ERR_INVALID_ARG;
  if (groups > RD_MAX_EXPERT_GROUPS) return RD_ERR_UNSUPPORTED;
  if (tokens > 0 && (ids == nullptr || weights == nullptr)) return RD_ERR_INVALID_ARG;
  if (!aligned4(bias) || !aligned4(ids) || !aligned4(weights)) return RD_ERR_UNSUPPORTED;
  const bool plan = group_sizes != nullptr || pos != nullptr || rows != nullptr;
  if (plan && (st = check_sort(tokens, config->topk, experts, ids, limit, group_sizes, pos, rows)) != RD_OK)
    return st;
  const uint64_t sb = static_cast<uint64_t>(tokens) * config->topk * 4, eb = static_cast<uint64_t>(experts) * 4;
  if (any_overlap<5, 3>({{ids, sb}, {weights, sb}, {group_sizes, eb}, {pos, sb}, {rows, 4}},
                        {{logits, static_cast<uint64_t>(tokens) * experts * (dtype == RD_F32 ? 4 : 2)},
                         {bias, eb},
                         {limit, 4}}))
    return RD_ERR_INVALID_ARG;
  int sms = 0;
  if ((st = current_device(&sms)) != RD_OK) return st;
  if (tokens > 0) {
    RouteArgs a = route_args(logits, config, tokens, experts, limit);
    a.bias = bias;
    a.ids = ids;
    a.weights = weights;
    if ((st = done(launch_route(a, dtype, sms, cu(stream)))) != RD_OK) return st;
  }
  if (!plan) return RD_OK;
  return done(launch_sort_rows(ids, static_cast<int32_t>(tokens), config->topk,
                               static_cast<int32_t>(experts), limit, group_sizes, pos, rows, cu(stream)));
}

extern "C" rd_status rd_route_bwd(const void* logits, int32_t dtype, const int32_t* ids,
                                  const float* d_weights, int64_t tokens, int64_t experts,
                                  const rd_route_config* config, const int32_t* limit,
                                  void* d_logits, rd_stream_t stream) {
  rd_status st = check_route(logits, dtype, tokens, experts, config, limit);
  if (st != RD_OK) return st;
  if (tokens > 0 && (ids == nullptr || d_weights == nullptr || d_logits == nullptr))
    return RD_ERR_INVALID_ARG;
  if (!aligned4(ids) || !aligned4(d_weights) ||
      (reinterpret_cast<uintptr_t>(d_logits) & (dtype == RD_F32 ? 3u : 1u)))
    return RD_ERR_UNSUPPORTED;
  const uint64_t lb = static_cast<uint64_t>(tokens) * experts * (dtype == RD_F32 ? 4 : 2);
  const uint64_t sb = static_cast<uint64_t>(tokens) * config->topk * 4;
  if (any_overlap<1, 4>({{d_logits, lb}}, {{logits, lb}, {ids, sb}, {d_weights, sb}, {limit, 4}}))
    return RD_ERR_INVALID_ARG;
  int sms = 0;
  if ((st = current_device(&sms)) != RD_OK) return st;
  if (tokens == 0) return RD_OK;
  RouteArgs a = route_args(logits, config, tokens, experts, limit);
  a.ids = const_cast<int32_t*>(ids);
  a.d_weights = d_weights;
  a.d_logits = d_logits;
  return done(launch_route_bwd(a, dtype, sms, cu(stream)));
}

extern "C" rd_status rd_sort_rows(const int32_t* ids, int64_t tokens, int64_t topk, int64_t experts,
                                  const int32_t* limit, int32_t* group_sizes, int32_t* pos,
                                  int32_t* rows, rd_stream_t stream) {
  rd_status st = check_sort(tokens, topk, experts, ids, limit, group_sizes, pos, rows);
  if (st != RD_OK) return st;
  const uint64_t sb = static_cast<uint64_t>(tokens) * topk * 4, eb = static_cast<uint64_t>(experts) * 4;
  if (any_overlap<3, 2>({{group_sizes, eb}, {pos, sb}, {rows, 4}}, {{ids, sb}, {limit, 4}}))
    return RD_ERR_INVALID_ARG;
  int sms = 0;
  if ((st = current_device(&sms)) != RD_OK) return st;
  return done(launch_sort_rows(ids, static_cast<int32_t>(tokens), static_cast<int32_t>(topk),
                               static_cast<int32_t>(experts), limit, group_sizes, pos, rows, cu(stream)));
}

namespace {

// checks of the three row movers: matrix a is [tokens, hidden], matrix b [packed_rows, hidden]
rd_status check_rows(const void* a, const void* b, const int32_t* pos, const int32_t* limit,
                     int64_t tokens, int64_t topk, int64_t hidden, int64_t packed_rows) {
  if (tokens < 0 || topk < 1 || hidden < 0 || packed_rows < 0) return RD_ERR_INVALID_ARG;
  if (topk > RD_MAX_TOPK || tokens > kMaxDim || hidden > kMaxDim || packed_rows > kMaxDim ||
      tokens * topk > kMaxDim || hidden % 8 != 0)
    return RD_ERR_UNSUPPORTED;
  if (tokens > 0 && pos == nullptr) return RD_ERR_INVALID_ARG;
  if ((tokens > 0 && hidden > 0 && a == nullptr) || (packed_rows > 0 && hidden > 0 && b == nullptr))
    return RD_ERR_INVALID_ARG;
  if (!aligned16(a) || !aligned16(b) || !aligned4(pos) || !aligned4(limit)) return RD_ERR_UNSUPPORTED;
  return RD_OK;
}

RowsArgs rows_args(const int32_t* pos, const int32_t* limit, int64_t tokens, int64_t topk,
                   int64_t hidden, int64_t packed_rows) {
  RowsArgs a = {};
  a.pos = pos;
  a.limit = limit;
  a.tokens = static_cast<int32_t>(tokens);
  a.topk = static_cast<int32_t>(topk);
  a.vecs = static_cast<int32_t>(hidden / 8);
  a.packed_rows = static_cast<int32_t>(packed_rows);
  return a;
}

}  // namespace

extern "C" rd_status rd_dispatch_rows(const void* x, const int32_t* pos, void* out, int64_t tokens,
                                      int64_t topk, int64_t hidden, int64_t out_rows,
                                      const int32_t* limit, rd_stream_t stream) {
  rd_status st = check_rows(x, out, pos, limit, tokens, topk, hidden, out_rows);
  if (st != RD_OK) return st;
  if (any_overlap<1, 3>({{out, static_cast<uint64_t>(out_rows) * hidden * 2}},
                        {{x, static_cast<uint64_t>(tokens) * hidden * 2},
                         {pos, static_cast<uint64_t>(tokens) * topk * 4},
                         {limit, 4}}))
    return RD_ERR_INVALID_ARG;
  int sms = 0;
  if ((st = current_device(&sms)) != RD_OK) return st;
  if (tokens == 0 || hidden == 0 || out_rows == 0) return RD_OK;
  RowsArgs a = rows_args(pos, limit, tokens, topk, hidden, out_rows);
  a.x = x;
  a.out = out;
  return done(launch_dispatch_rows(a, sms, cu(stream)));
}

extern "C" rd_status rd_combine_rows(const void* y, const int32_t* pos, const float* w, void* out,
                                     int64_t tokens, int64_t topk, int64_t hidden, int64_t y_rows,
                                     const int32_t* limit, rd_stream_t stream) {
  rd_status st = check_rows(out, y, pos, limit, tokens, topk, hidden, y_rows);
  if (st != RD_OK) return st;
  if (!aligned4(w)) return RD_ERR_UNSUPPORTED;
  const uint64_t sb = static_cast<uint64_t>(tokens) * topk * 4;
  if (any_overlap<1, 4>({{out, static_cast<uint64_t>(tokens) * hidden * 2}},
                        {{y, static_cast<uint64_t>(y_rows) * hidden * 2}, {pos, sb}, {w, sb}, {limit, 4}}))
    return RD_ERR_INVALID_ARG;
  int sms = 0;
  if ((st = current_device(&sms)) != RD_OK) return st;
  if (tokens == 0 || hidden == 0) return RD_OK;
  RowsArgs a = rows_args(pos, limit, tokens, topk, hidden, y_rows);
  a.x = y;
  a.w = w;
  a.out = out;
  return done(launch_combine_rows(a, sms, cu(stream)));
}

extern "C" rd_status rd_combine_rows_bwd(const void* d_out, const void* y, const int32_t* pos,
                                         const float* w, void* d_y, float* d_w, int64_t tokens,
                                         int64_t topk, int64_t hidden, int64_t y_rows,
                                         const int32_t* limit, rd_stream_t stream) {
  rd_status st = check_rows(d_out, y, pos, limit, tokens, topk, hidden, y_rows);
  if (st != RD_OK) return st;
  if (tokens > 0 && (w == nullptr || d_w == nullptr)) return RD_ERR_INVALID_ARG;
  if (y_rows > 0 && hidden > 0 && d_y == nullptr) return RD_ERR_INVALID_ARG;
  if (!aligned16(d_y) || !aligned4(w) || !aligned4(d_w)) return RD_ERR_UNSUPPORTED;
  const uint64_t sb = static_cast<uint64_t>(tokens) * topk * 4;
  const uint64_t yb = static_cast<uint64_t>(y_rows) * hidden * 2;
  if (any_overlap<2, 5>({{d_y, yb}, {d_w, sb}},
                        {{d_out, static_cast<uint64_t>(tokens) * hidden * 2}, {y, yb}, {pos, sb}, {w, sb}, {limit, 4}}))
    return RD_ERR_INVALID_ARG;
  int sms = 0;
  if ((st = current_device(&sms)) != RD_OK) return st;
  if (tokens == 0) return RD_OK;
  RowsArgs a = rows_args(pos, limit, tokens, topk, hidden, y_rows);
  a.x = d_out;
  a.y = y;
  a.w = w;
  a.out = d_y;
  a.d_w = d_w;
  return done(launch_combine_rows_bwd(a, sms, cu(stream)));
}

// ------------------------------------------------------------------ 4-bit rows
extern "C" int64_t rd_mxfp4_scale_width(int64_t k) { return k <= 0 ? 0 : (k / 32 + 15) / 16 * 16; }

namespace {

// x [rows, k], q and scales of q_rows rows
rd_status check_mx(const void* x, const void* q, const void* scales, int64_t rows, int64_t q_rows,
                   int64_t k, const int32_t* limit) {
  if (rows < 0 || q_rows < 0 || k < 0) return RD_ERR_INVALID_ARG;
  if (rows > kMaxDim || q_rows > kMaxDim || k > kMaxDim || k % 32 != 0) return RD_ERR_UNSUPPORTED;
  if (rows > 0 && k > 0 && (x == nullptr || (q_rows > 0 && (q == nullptr || scales == nullptr))))
    return RD_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(q) || !aligned16(scales) || !aligned4(limit)) return RD_ERR_UNSUPPORTED;
  return RD_OK;
}

}  // namespace

extern "C" rd_status rd_mxfp4_quantize(const void* x, const int32_t* pos, void* q, void* scales,
                                       int64_t rows, int64_t topk, int64_t k, int64_t out_rows,
                                       const int32_t* limit, rd_stream_t stream) {
  rd_status st = check_mx(x, q, scales, rows, out_rows, k, limit);
  if (st != RD_OK) return st;
  if (pos == nullptr) {
    if (out_rows < rows) return RD_ERR_INVALID_ARG;
    topk = 1;
  } else {
    if (topk < 1) return RD_ERR_INVALID_ARG;
    if (topk > RD_MAX_TOPK || rows * topk > kMaxDim || !aligned4(pos)) return RD_ERR_UNSUPPORTED;
  }
  const int64_t width = rd_mxfp4_scale_width(k);
  if (any_overlap<2, 3>({{q, static_cast<uint64_t>(out_rows) * (k / 2)},
                         {scales, static_cast<uint64_t>(out_rows) * width}},
                        {{x, static_cast<uint64_t>(rows) * k * 2},
                         {pos, static_cast<uint64_t>(rows) * topk * 4},
                         {limit, 4}}))
    return RD_ERR_INVALID_ARG;
  int sms = 0;
  if ((st = current_device(&sms)) != RD_OK) return st;
  if (rows == 0 || k == 0 || out_rows == 0) return RD_OK;
  QuantArgs a = {};
  a.x = x;
  a.pos = pos;
  a.q = static_cast<uint8_t*>(q);
  a.scales = static_cast<uint8_t*>(scales);
  a.limit = limit;
  a.rows = static_cast<int32_t>(rows);
  a.topk = static_cast<int32_t>(topk);
  a.k = static_cast<int32_t>(k);
  a.scale_width = static_cast<int32_t>(width);
  a.out_rows = static_cast<int32_t>(out_rows);
  return done(launch_mxfp4_quantize(a, sms, cu(stream)));
}

extern "C" rd_status rd_mxfp4_dequantize(const void* q, const void* scales, void* out, int64_t rows,
                                         int64_t k, const int32_t* limit, rd_stream_t stream) {
  rd_status st = check_mx(out, q, scales, rows, rows, k, limit);
  if (st != RD_OK) return st;
  const int64_t width = rd_mxfp4_scale_width(k);
  if (any_overlap<1, 3>({{out, static_cast<uint64_t>(rows) * k * 2}},
                        {{q, static_cast<uint64_t>(rows) * (k / 2)},
                         {scales, static_cast<uint64_t>(rows) * width},
                         {limit, 4}}))
    return RD_ERR_INVALID_ARG;
  int sms = 0;
  if ((st = current_device(&sms)) != RD_OK) return st;
  if (rows == 0 || k == 0) return RD_OK;
  QuantArgs a = {};
  a.q = const_cast<uint8_t*>(static_cast<const uint8_t*>(q));
  a.scales = const_cast<uint8_t*>(static_cast<const uint8_t*>(scales));
  a.limit = limit;
  a.rows = static_cast<int32_t>(rows);
  a.k = static_cast<int32_t>(k);
  a.scale_width = static_cast<int32_t>(width);
  return done(launch_mxfp4_dequantize(a, out, sms, cu(stream)));
}

extern "C" rd_status rd_mxfp4_quantize_weights(const void* rhs, void* q, void* scales, int64_t g,
                                               int64_t k, int64_t n, rd_stream_t stream) {
  if (g < 0 || k < 0 || n < 0) return RD_ERR_INVALID_ARG;
  // the launch spans g and the scale bytes of a row in grid dimensions of at most 65535
  if (g > 65535 || k > 32 * int64_t{65520} || n > kMaxDim || k % 32 != 0 || n % 8 != 0)
    return RD_ERR_UNSUPPORTED;
  const bool any = g > 0 && k > 0 && n > 0;
  if (any && (rhs == nullptr || q == nullptr || scales == nullptr)) return RD_ERR_INVALID_ARG;
  if (!aligned16(rhs) || !aligned16(q) || !aligned16(scales)) return RD_ERR_UNSUPPORTED;
  const int64_t width = rd_mxfp4_scale_width(k);
  const uint64_t rows = static_cast<uint64_t>(g) * n;
  if (any_overlap<2, 1>({{q, rows * (k / 2)}, {scales, rows * width}}, {{rhs, rows * k * 2}}))
    return RD_ERR_INVALID_ARG;
  int sms = 0;
  rd_status st = current_device(&sms);
  if (st != RD_OK) return st;
  if (!any) return RD_OK;
  return done(launch_mxfp4_quantize_weights(rhs, static_cast<uint8_t*>(q), static_cast<uint8_t*>(scales),
                                            static_cast<int32_t>(g), static_cast<int32_t>(k),
                                            static_cast<int32_t>(n), static_cast<int32_t>(width),
                                            cu(stream)));
}

extern "C" rd_status rd_ragged_dot_mxfp4(const void* a, const void* a_scales, const void* b,
                                         const void* b_scales, void* out, void* out_scales,
                                         int64_t m, int64_t k, int64_t n,
                                         const int32_t* group_sizes, int32_t g_total,
                                         int32_t group_offset, int32_t g_local,
                                         const int32_t* limit, int32_t epi, int32_t* status,
                                         rd_stream_t stream) {
  if (epi != RD_EPI_NONE && epi != RD_EPI_SILU_GLU && epi != RD_EPI_SILU_GLU_MXFP4)
    return RD_ERR_INVALID_ARG;
  rd_status st = check_groups(m, k, n, group_sizes, g_total, group_offset, g_local, limit, status);
  if (st != RD_OK) return st;
  const bool glu = epi != RD_EPI_NONE, quant = epi == RD_EPI_SILU_GLU_MXFP4;
  if (k % 32 != 0) return RD_ERR_UNSUPPORTED;
  if (glu && n % (quant ? 64 : 16) != 0) return RD_ERR_UNSUPPORTED;
  const int64_t n_out = glu ? n / 2 : n;
  // the kernel counts k in 32 bits, up to a shared-memory slot of scales past its end
  if (n_out > kMaxWidth || k > kMaxDim + 1 - k4RawK) return RD_ERR_UNSUPPORTED;
  if ((m > 0 && k > 0 && (a == nullptr || a_scales == nullptr)) ||
      (k > 0 && n > 0 && (b == nullptr || b_scales == nullptr)) ||
      (m > 0 && n > 0 && (out == nullptr || quant != (out_scales != nullptr))))
    return RD_ERR_INVALID_ARG;
  if (!aligned16(a) || !aligned16(a_scales) || !aligned16(b) || !aligned16(b_scales) ||
      !aligned16(out) || !aligned16(out_scales))
    return RD_ERR_UNSUPPORTED;
  const uint64_t um = static_cast<uint64_t>(m), ug = static_cast<uint64_t>(g_local);
  const int64_t width = rd_mxfp4_scale_width(k), out_width = quant ? rd_mxfp4_scale_width(n_out) : 0;
  if (any_overlap<2, 7>({{out, quant ? um * (n_out / 2) : um * n_out * 2}, {out_scales, um * out_width}},
                        {{a, um * (k / 2)},
                         {a_scales, um * width},
                         {b, ug * n * (k / 2)},
                         {b_scales, ug * n * width},
                         {group_sizes, static_cast<uint64_t>(g_total) * 4},
                         {limit, 4},
                         {status, 4}}))
    return RD_ERR_INVALID_ARG;
  int sms = 0;
  if ((st = current_device(&sms)) != RD_OK) return st;
  if (m == 0 || n == 0) return RD_OK;

  // Tiles of 32 rows where the groups average at most 16 (most of them then hold a tile's rows or fewer; see
  // gemm_mxfp4.cuh), of 256 on CTA pairs from 512 on (use_pair), of 128 between.  By rows a group, us:
  //                                        1     16     24     32     48    192    256    512   1024
  //   4096 -> 1536, 128 experts    32    47.0   69.3   69.7   72.0   88.9
  //                               128    48.4   70.2   70.8   71.3   72.3  103.7  120.1  202.5  379.7
  //                               256    54.0   81.6   82.2   82.8   83.5   90.7  119.7  182.4  327.6
  //   768 -> 4096, 128 experts     32    29.8   41.5   42.9   47.8   63.3
  //                               128    37.7   42.3   43.1   43.8   46.0   81.9   95.2  162.4  299.8
  //                               256    53.1   65.1   65.5   59.8   61.7   80.7  111.0  168.4  298.4
  //   4096 -> 14336, 8 experts     32    33.7   42.6   42.9   47.6   49.9
  //                               128    38.6   43.7   44.2   44.2   44.6   63.5   72.5  116.2  208.4
  //                               256    61.1   50.4   51.1   51.1   51.8   55.4   70.9  106.6  181.1
  // 32 against 128: the sides meet between 24 and 32.  128 against 256: at k = 4096 pairs are ahead from 192
  // rows on (by up to 14 %; even at 256), at k = 768 they are behind at 256 and 512 and even at 1024.  The bf16
  // products' 512 lies between the two.
  const bool pair = use_pair(sms, m, g_total);
  const bool few = !pair && m <= 16 * static_cast<int64_t>(g_total);
  const int tm = pair ? 2 * kBM : (few ? 32 : kBM);
  Gemm4Maps maps = {};
  if (k > 0) {
    // rows of k / 2 bytes as k / 4 two-byte elements, boxes of 128 bytes of a row; scale rows as
    // width / 2 such elements, boxes of 32 bytes
    const uint64_t da[2] = {static_cast<uint64_t>(k / 4), um};
    const uint64_t sa[1] = {static_cast<uint64_t>(k / 2)};
    const uint32_t a_rows = few ? 32 : kBM;
    const uint32_t ba[2] = {64, a_rows};
    if ((st = encode(&maps.a, a, 2, da, sa, ba)) != RD_OK) return st;
    const uint64_t db[3] = {static_cast<uint64_t>(k / 4), static_cast<uint64_t>(n), ug};
    const uint64_t sb[2] = {static_cast<uint64_t>(k / 2), static_cast<uint64_t>(n) * (k / 2)};
    const uint32_t bb[3] = {64, k4Half, 1};
    if ((st = encode(&maps.b, b, 3, db, sb, bb)) != RD_OK) return st;
    const uint64_t w = static_cast<uint64_t>(width);
    const uint64_t das[2] = {w / 2, um}, sas[1] = {w};
    const uint32_t bas[2] = {16, a_rows};
    if ((st = encode(&maps.a_scales, a_scales, 2, das, sas, bas, CU_TENSOR_MAP_SWIZZLE_32B)) != RD_OK)
      return st;
    const uint64_t dbs[3] = {w / 2, static_cast<uint64_t>(n), ug}, sbs[2] = {w, static_cast<uint64_t>(n) * w};
    const uint32_t bbs[3] = {16, k4Half, 1};
    if ((st = encode(&maps.b_scales, b_scales, 3, dbs, sbs, bbs, CU_TENSOR_MAP_SWIZZLE_32B)) != RD_OK)
      return st;
  }
  const int tile_w = glu ? k4Half : k4BN;
  Gemm4Args g = {};
  g.group_sizes = group_sizes;
  g.limit = limit;
  g.status = status;
  g.out = out;
  g.out_scales = static_cast<uint8_t*>(out_scales);
  g.m = static_cast<int32_t>(m);
  g.kc = static_cast<int32_t>(k);
  g.n_out = static_cast<int32_t>(n_out);
  g.out_scale_width = static_cast<int32_t>(out_width);
  g.g_total = g_total;
  g.group_offset = group_offset;
  g.g_local = g_local;
  g.n_tiles = static_cast<int32_t>((n_out + tile_w - 1) / tile_w);
  // a 4-bit row is a quarter of a bf16 row: bands of four times the rows keep as many bytes in L2
  // (32768 x 4096 x 14336: 623 -> 617 us, means of six)
  g.band_tiles = band_tiles(pair, 4 * kBandRows) * (few ? kBM / 32 : 1);
  g.wait = wait_limit();
  const int64_t tiles = ((m + tm - 1) / tm + g_local) * g.n_tiles;
  if (tiles > kMaxDim) return RD_ERR_UNSUPPORTED;
  const int grid = pair ? pair_grid(sms, tiles) : grid_for(sms, tiles);
  const int which = quant ? k4EpiGluQuant : (glu ? k4EpiGlu : k4EpiNone);
  return done(launch_gemm_mxfp4(which, pair ? k4Pair : (few ? k4Few : k4Single), maps, g, grid, cu(stream)));
}
