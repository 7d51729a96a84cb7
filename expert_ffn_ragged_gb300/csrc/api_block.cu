// api_block.cu -- the C entry points of include/rd_block.h: argument checks (all of those that the
// host can make come before any CUDA call), tensor maps, launch shapes.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/rd_block.h"
#include "block_args.h"
#include "gemm_args.h"
#include "gemm_split.h"
#include "host.h"

using namespace rd;

namespace {

rd_status done(cudaError_t e) { return e == cudaSuccess ? RD_OK : RD_ERR_CUDA; }

cudaStream_t cu(rd_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

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

bool known(int32_t dtype) { return dtype == RD_F32 || dtype == RD_BF16; }
uint64_t size_of(int32_t dtype) { return dtype == RD_F32 ? 4 : 2; }
// matrices: 16 bytes, f32 ones 32 (eight elements are one access)
bool matrix_aligned(const void* p, int32_t dtype) {
  return (reinterpret_cast<uintptr_t>(p) & (dtype == RD_F32 ? 31u : 15u)) == 0;
}

rd_status check_matrix(int64_t rows, int64_t hidden, int32_t dtype, int32_t out_dtype) {
  if (rows < 0 || hidden < 0 || !known(dtype) || !known(out_dtype)) return RD_ERR_INVALID_ARG;
  if (rows > kMaxDim || hidden > kMaxDim || hidden % 8 != 0) return RD_ERR_UNSUPPORTED;
  return RD_OK;
}

}  // namespace

extern "C" rd_status rd_layer_norm_fwd(const void* x, int32_t dtype, const float* weight,
                                       const float* bias, float eps, void* out, int32_t out_dtype,
                                       float* mean, float* rstd, int64_t rows, int64_t hidden,
                                       const int32_t* limit, rd_stream_t stream) {
  rd_status st = check_matrix(rows, hidden, dtype, out_dtype);
  if (st == RD_ERR_INVALID_ARG) return st;
  if (!(eps >= 0.0f) || isinf(eps) || (mean == nullptr) != (rstd == nullptr)) return RD_ERR_INVALID_ARG;
  if (rows > 0 && hidden > 0 && (x == nullptr || out == nullptr)) return RD_ERR_INVALID_ARG;
  if (st != RD_OK) return st;
  if (!matrix_aligned(x, dtype) || !matrix_aligned(out, out_dtype) || !aligned16(weight) || !aligned16(bias) ||
      !aligned4(mean) || !aligned4(rstd) || !aligned4(limit))
    return RD_ERR_UNSUPPORTED;
  const uint64_t n = static_cast<uint64_t>(rows) * hidden, rb = static_cast<uint64_t>(rows) * 4,
                 hb = static_cast<uint64_t>(hidden) * 4;
  if (any_overlap<3, 4>({{out, n * size_of(out_dtype)}, {mean, rb}, {rstd, rb}},
                        {{x, n * size_of(dtype)}, {weight, hb}, {bias, hb}, {limit, 4}}))
    return RD_ERR_INVALID_ARG;
  int sms = 0;
  if ((st = current_device(&sms)) != RD_OK) return st;
  if (rows == 0 || hidden == 0) return RD_OK;
  NormArgs a = {};
  a.x = x;
  a.weight = weight;
  a.bias = bias;
  a.out = out;
  a.mean = mean;
  a.rstd = rstd;
  a.limit = limit;
  a.rows = static_cast<int32_t>(rows);
  a.hidden = static_cast<int32_t>(hidden);
  a.eps = eps;
  return done(launch_layer_norm_fwd(a, dtype, out_dtype, sms, cu(stream)));
}

namespace {
uint64_t norm_bwd_bytes(int64_t rows, int64_t hidden, int sms) {
  return static_cast<uint64_t>(layer_norm_bwd_parts(rows, hidden, sms)) * 2 * static_cast<uint64_t>(hidden) * 4;
}
}  // namespace

extern "C" rd_status rd_layer_norm_bwd_workspace_size(int64_t rows, int64_t hidden, size_t* bytes) {
  if (bytes == nullptr) return RD_ERR_INVALID_ARG;
  rd_status st = check_matrix(rows, hidden, RD_F32, RD_F32);
  if (st != RD_OK) return st;
  int sms = 0;
  if ((st = current_device(&sms)) != RD_OK) return st;
  *bytes = norm_bwd_bytes(rows, hidden, sms);
  return RD_OK;
}

extern "C" rd_status rd_layer_norm_bwd(const void* d_out, int32_t out_dtype, const void* x,
                                       int32_t dtype, const float* weight, const float* mean,
                                       const float* rstd, void* d_x, float* d_weight, float* d_bias,
                                       int64_t rows, int64_t hidden, const int32_t* limit,
                                       void* workspace, size_t workspace_bytes, rd_stream_t stream) {
  rd_status st = check_matrix(rows, hidden, dtype, out_dtype);
  if (st == RD_ERR_INVALID_ARG) return st;
  const bool sums = d_weight != nullptr || d_bias != nullptr;
  if (rows > 0 && hidden > 0 &&
      (x == nullptr || d_out == nullptr || d_x == nullptr || mean == nullptr || rstd == nullptr))
    return RD_ERR_INVALID_ARG;
  if (sums && hidden > 0 && workspace == nullptr && !layer_norm_bwd_few(rows, hidden)) return RD_ERR_INVALID_ARG;
  if (st != RD_OK) return st;
  if (!matrix_aligned(x, dtype) || !matrix_aligned(d_x, dtype) || !matrix_aligned(d_out, out_dtype) ||
      !aligned16(weight) || !aligned16(d_weight) || !aligned16(d_bias) || !matrix_aligned(workspace, RD_F32) ||
      !aligned4(mean) ||
      !aligned4(rstd) || !aligned4(limit))
    return RD_ERR_UNSUPPORTED;
  const uint64_t n = static_cast<uint64_t>(rows) * hidden, rb = static_cast<uint64_t>(rows) * 4,
                 hb = static_cast<uint64_t>(hidden) * 4;
  if (any_overlap<4, 6>({{d_x, n * size_of(dtype)}, {d_weight, hb}, {d_bias, hb}, {sums ? workspace : nullptr, workspace_bytes}},
                        {{x, n * size_of(dtype)}, {d_out, n * size_of(out_dtype)}, {weight, hb}, {mean, rb}, {rstd, rb}, {limit, 4}}))
    return RD_ERR_INVALID_ARG;
  int sms = 0;
  if ((st = current_device(&sms)) != RD_OK) return st;
  const uint64_t need = sums && hidden > 0 ? norm_bwd_bytes(rows, hidden, sms) : 0;
  if (workspace_bytes < need) return RD_ERR_INVALID_ARG;
  if (hidden == 0) return RD_OK;
  if (rows == 0 && !sums) return RD_OK;
  NormArgs a = {};
  a.x = x;
  a.d_out = d_out;
  a.weight = weight;
  a.out = d_x;
  a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.d_weight = d_weight;
  a.d_bias = d_bias;
  a.parts = need > 0 ? static_cast<float*>(workspace) : nullptr;
  a.wait = wait_limit();
  a.limit = limit;
  a.rows = static_cast<int32_t>(rows);
  a.hidden = static_cast<int32_t>(hidden);
  return done(launch_layer_norm_bwd(a, dtype, out_dtype, sms, cu(stream)));
}

extern "C" rd_status rd_dropout_rows(const void* x, int32_t dtype, const void* residual,
                                     const int64_t* rng, float p, void* out, int32_t out_dtype,
                                     int64_t rows, int64_t hidden, const int32_t* limit,
                                     rd_stream_t stream) {
  rd_status st = check_matrix(rows, hidden, dtype, out_dtype);
  if (st == RD_ERR_INVALID_ARG) return st;
  if (!(p >= 0.0f && p <= 1.0f) || rng == nullptr) return RD_ERR_INVALID_ARG;
  if (rows > 0 && hidden > 0 && (x == nullptr || out == nullptr)) return RD_ERR_INVALID_ARG;
  if (st != RD_OK) return st;
  if (!matrix_aligned(x, dtype) || !matrix_aligned(out, out_dtype) || !matrix_aligned(residual, out_dtype) ||
      (reinterpret_cast<uintptr_t>(rng) & 7u) || !aligned4(limit))
    return RD_ERR_UNSUPPORTED;
  const uint64_t n = static_cast<uint64_t>(rows) * hidden;
  if (any_overlap<1, 4>({{out, n * size_of(out_dtype)}},
                        {{x, n * size_of(dtype)}, {residual, n * size_of(out_dtype)}, {rng, 16}, {limit, 4}}))
    return RD_ERR_INVALID_ARG;
  int sms = 0;
  if ((st = current_device(&sms)) != RD_OK) return st;
  if (rows == 0 || hidden == 0) return RD_OK;
  DropoutArgs a = {};
  a.x = x;
  a.residual = residual;
  a.out = out;
  a.rng = rng;
  a.limit = limit;
  a.rows = static_cast<int32_t>(rows);
  a.vecs = static_cast<int32_t>(hidden / 8);
  a.least = static_cast<int32_t>(floor(static_cast<double>(p) * 65536.0 + 0.5));
  a.scale = a.least < 65536 ? static_cast<float>(65536.0 / (65536 - a.least)) : 0.0f;
  return done(launch_dropout_rows(a, dtype, out_dtype, sms, cu(stream)));
}

// ------------------------------------------------------------------ products with an epilogue
namespace {

// the checks that rd_linear and its gradient share; without group sizes there is one group of all rows
rd_status check_linear(int64_t m, int64_t k, int64_t n, const int32_t* group_sizes, int32_t g_total,
                       int32_t group_offset, int32_t g_local, const int32_t* limit,
                       const int32_t* status, int32_t act, int32_t out_dtype) {
  if (act < RD_ACT_NONE || act > RD_ACT_SILU || !known(out_dtype)) return RD_ERR_INVALID_ARG;
  static const int32_t none = 0;
  if (group_sizes == nullptr && (g_total != 1 || group_offset != 0 || g_local != 1)) return RD_ERR_INVALID_ARG;
  rd_status st = check_groups(m, k, n, group_sizes != nullptr ? group_sizes : &none, g_total, group_offset, g_local,
                              limit, status);
  if (st != RD_OK) return st;
  return n > kMaxWidth ? RD_ERR_UNSUPPORTED : RD_OK;
}

// Rows of an output tile of the kernel that splits k.  By group a tile is two to four times as high as the average group.
int32_t split_rows(int64_t m, bool groups, int32_t g_total) {
  int64_t rows = kSplitRows;
  if (groups)
    while (rows > 8 && rows / 2 * g_total >= 2 * m) rows /= 2;
  return static_cast<int32_t>(m < rows ? (m + 7) / 8 * 8 : rows);
}

// The most row tiles that there can be: by group, a last tile that is not full for every group with rows.
int64_t most_row_tiles(int64_t m, int32_t rows, bool groups, int32_t g_local) {
  return groups ? (m < g_local ? m : g_local) + m / rows : (m + rows - 1) / rows;
}
// As many as the rules below reckon with: by group, one each or, of long groups, half a tile that is not full.
int64_t usual_row_tiles(int64_t m, int32_t rows, bool groups, int32_t g_local) {
  const int64_t most = most_row_tiles(m, rows, groups, g_local), some = m < g_local ? m : g_local;
  return groups ? (most - g_local / 2 > some ? most - g_local / 2 : some) : most;
}

// Few tiles: the kernel that splits k over clusters, or the persistent one, whose tiles are twice as wide (and on
// CTA pairs twice as high).  At k = 4096, us split / persistent:
//   m x n     16 x 14336  512 x 4096  2048 x 1024  16381 x 128  2500 x 1024  256 x 14336  1024 x 4096  16384 x 256
//   tiles     112         128         128          128          160          224          256          256
//             22 / 37     20 / 29     21 / 29      30 / 35      32 / 28      38 / 37      32 / 29      37 / 34
// and by group (rows x k x n, groups): 4 x 2960 x 392, 16: 7.4 / 31; 310 x 2912 x 64, 4: 7.1 / 19; 128 x 4096 x 1024, 8: 18 / 35;
// 8 x 7168 x 2048, 32: 39 / 62; 4096 x 1024 x 256, 16: 12 / 19.  A short k leaves the persistent kernel's few epilogue warps too much of the
// time (200 to 256 tiles, n = 1024, k = 512 / 1024 / 2048: 10 / 13, 14 / 15, 20 / 19; f32 14.4 / 15.0, 19.6 / 17.4; 30000 x 512 x 128 12 / 17),
// except by group in f32 (100 x 512 x 512 in 128 groups 20 / 15).
bool use_split(int sms, int64_t wide, int64_t k, bool groups, bool f32) {
  const bool brief = k <= (f32 ? 512 : 1024) && !(groups && f32);
  return wide <= (brief ? 3 : 1) * static_cast<int64_t>(sms);
}

// By group also where there are more tiles but few rows a group: the weights are the time, and its tiles are half as wide, so that they
// spread better over the SMs, if they do not take many turns (bf16, us split / persistent: 16 x 4096 x 4096 in 8 groups 36 / 39, 607 x 1280 x 2176
// in 16 21 / 23, 256 x 2048 x 1024 in 64 45 / 47, 32 x 7168 x 2048 in 32 106 / 122, 8 x 2048 x 7168 in 32 40 / 50, but 512 x 4096 x 4096 in 8 48 /
// 49, 4096 x 2048 x 1024 in 64 56 / 52, and with 896 tiles 64 x 4096 x 14336 in 8 147 / 142).  Its f32 tiles of 64 columns that run in
// turns are slower (512 x 4096 x 4096 in 8: 59 / 52).
bool short_groups(int sms, int64_t m, int64_t wide, int32_t g_total, bool f32) {
  return !f32 && m <= 48 * static_cast<int64_t>(g_total) && wide <= 4 * static_cast<int64_t>(sms);
}

// Its tiles have 128 columns where these are tiles enough for more than half of the SMs, else 64 (tiles of 64 then have an SM each or
// share their k).  At k = 4096, us 64 / 128:
//   m x n     256 x 4096  4096 x 256  64 x 4096 (k = 14336)  1 x 11264  384 x 4096  11000 x 128  1 x 14336  512 x 4096  256 x 14336
//   tiles     64          64          32                     88         96          86           112        128         224
//             17 / 20     17 / 20     25 / 29                21 / 20    24 / 21     27 / 24      24 / 23    24 / 23     53 / 39
// An f32 output of 128 columns holds a row's sums in so many registers that its CTA has the SM for itself.
int split_cols(int sms, int64_t wide, bool f32) {
  return 2 * wide > static_cast<int64_t>(sms) && (!f32 || wide <= sms) ? 128 : 64;
}

// Where tiles of 128 columns are more than half of the SMs and no more than all, each has an SM and a deep ring for
// itself (us against two CTAs a tile on half the ring, k = 4096: 1 x 14336 21.6 / 22.2, 96 x 14336 25.8 / 27.4, 16381 x 128
// 30.6 / 31.9).  Otherwise as many CTAs a tile as still all run at once, two on an SM, with at least four K blocks each
// (tiles of 64 columns, 256 x 4096: 16.3 on two CTAs a tile, 19.8 alone; 64 x 4096, k = 14336: 23.9 on four, 33 on two
// with the deep ring).
bool split_alone(int sms, int cols, int64_t tiles) { return cols == 128 && tiles <= sms; }

int split_cluster(int sms, int cols, int64_t tiles, int64_t k) {
  if (cols == 128) return 1;  // tiles for more than half of the SMs
  const int64_t blocks = (k + kBK - 1) / kBK;
  int c = 1;
  while (c < 8 && tiles * c <= sms && blocks >= 8 * c) c *= 2;
  return c;
}

}  // namespace

extern "C" rd_status rd_linear(const void* x, const void* w, const float* bias, const void* residual,
                               int32_t act, void* out, int32_t out_dtype, void* pre, int64_t m,
                               int64_t k, int64_t n, const int32_t* group_sizes, int32_t g_total,
                               int32_t group_offset, int32_t g_local, const int32_t* limit,
                               int32_t* status, rd_stream_t stream) {
  rd_status st = check_linear(m, k, n, group_sizes, g_total, group_offset, g_local, limit, status, act, out_dtype);
  if (st != RD_OK) return st;
  if ((m > 0 && k > 0 && x == nullptr) || (k > 0 && n > 0 && w == nullptr) || (m > 0 && n > 0 && out == nullptr))
    return RD_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(w) || !aligned16(pre) || !aligned16(bias) || !matrix_aligned(out, out_dtype) ||
      !matrix_aligned(residual, out_dtype))
    return RD_ERR_UNSUPPORTED;
  const uint64_t um = static_cast<uint64_t>(m), ug = static_cast<uint64_t>(g_local), un = static_cast<uint64_t>(n);
  const uint64_t ob = um * un * size_of(out_dtype);
  if (any_overlap<2, 7>({{out, ob}, {pre, um * un * 2}},
                        {{x, um * k * 2},
                         {w, ug * k * un * 2},
                         {bias, ug * un * 4},
                         {residual, ob},
                         {group_sizes, static_cast<uint64_t>(g_total) * 4},
                         {limit, 4},
                         {status, 4}}))
    return RD_ERR_INVALID_ARG;
  int sms = 0;
  if ((st = current_device(&sms)) != RD_OK) return st;
  if (m == 0 || n == 0) return RD_OK;

  const bool groups = group_sizes != nullptr;
  const int32_t box_rows = split_rows(m, groups, g_total);
  const int64_t usual = usual_row_tiles(m, box_rows, groups, g_local), wide = usual * ((n + 127) / 128);
  const bool f32 = out_dtype == RD_F32;
  if (!(groups && variant_forced()) &&
      (use_split(sms, wide, k, groups, f32) || (groups && short_groups(sms, m, wide, g_total, f32)))) {
    const int cols = split_cols(sms, wide, f32);
    const int64_t tiles = usual * ((n + cols - 1) / cols);
    SplitArgs s = {};
    s.bias = bias;
    s.residual = residual;
    s.out = out;
    s.pre = pre;
    s.group_sizes = group_sizes;
    s.limit = limit;
    s.status = status;
    s.m = static_cast<int32_t>(m);
    s.k = static_cast<int32_t>(k);
    s.n = static_cast<int32_t>(n);
    s.act = act;
    s.g_total = g_total;
    s.group_offset = group_offset;
    s.g_local = g_local;
    s.box_rows = box_rows;
    s.row_tiles = static_cast<int32_t>(most_row_tiles(m, box_rows, groups, g_local));
    const int stage = s.box_rows * 128 + cols * kBK * 2;
    s.ring_bytes = split_alone(sms, cols, tiles) ? kSplitRingAlone : kSplitRing;
    s.stages = s.ring_bytes / stage < kSplitMaxStages ? s.ring_bytes / stage : kSplitMaxStages;
    s.cluster = split_cluster(sms, cols, tiles, k);
    s.wait = wait_limit();
    CUtensorMap tx = {}, tw = {};
    if (k > 0) {
      const uint64_t dx[2] = {static_cast<uint64_t>(k), um}, sx[1] = {static_cast<uint64_t>(k) * 2};
      const uint32_t bx[2] = {64, static_cast<uint32_t>(s.box_rows)};
      if ((st = encode(&tx, x, 2, dx, sx, bx)) != RD_OK) return st;
      const uint64_t dw[3] = {un, static_cast<uint64_t>(k), ug}, sw[2] = {un * 2, static_cast<uint64_t>(k) * un * 2};
      const uint32_t bw[3] = {64, kBK, 1};
      if ((st = encode(&tw, w, groups ? 3 : 2, dw, sw, bw)) != RD_OK) return st;
    }
    return done(launch_gemm_split(out_dtype == RD_F32, cols, tx, tw, s, cu(stream)));
  }

  const bool pair = use_pair(sms, m, g_total);
  CUtensorMap ta = {}, tb = {};
  if (k > 0) {
    const uint64_t da[2] = {static_cast<uint64_t>(k), um}, sa[1] = {static_cast<uint64_t>(k) * 2};
    const uint32_t ba[2] = {64, kBM};
    if ((st = encode(&ta, x, 2, da, sa, ba)) != RD_OK) return st;
    const uint64_t db[3] = {un, static_cast<uint64_t>(k), ug};
    const uint64_t sb[2] = {un * 2, static_cast<uint64_t>(k) * un * 2};
    const uint32_t bb[3] = {64, kBK, 1};
    if ((st = encode(&tb, w, 3, db, sb, bb)) != RD_OK) return st;
  }
  GemmArgs a = {};
  a.group_sizes = group_sizes;
  a.limit = limit;
  a.status = status;
  a.out = out;
  a.m = static_cast<int32_t>(m);
  a.kc = static_cast<int32_t>(k);
  a.n_out = static_cast<int32_t>(n);
  a.g_total = g_total;
  a.group_offset = group_offset;
  a.g_local = g_local;
  a.ldo = n;
  a.zero_cols = static_cast<int32_t>(n);
  a.n_tiles = static_cast<int32_t>((n + kBN - 1) / kBN);
  a.wait = wait_limit();
  a.band_tiles = band_tiles(pair);
  a.bias = bias;
  a.residual = residual;
  a.pre = pre;
  a.act = act;
  const int64_t tile = pair ? 2 * kBM : kBM;
  const int64_t tiles = ((m + tile - 1) / tile + g_local) * a.n_tiles;
  if (tiles > kMaxDim) return RD_ERR_UNSUPPORTED;
  const int grid = pair ? pair_grid(sms, tiles) : grid_for(sms, tiles);
  return done(launch_gemm_linear(out_dtype == RD_F32, pair, ta, tb, a, grid, cu(stream)));
}

extern "C" rd_status rd_linear_act_bwd_workspace_size(int64_t m, int64_t n, int32_t g_local, size_t* bytes) {
  if (bytes == nullptr || m < 0 || n < 0 || g_local < 1) return RD_ERR_INVALID_ARG;
  if (m > kMaxDim || n > kMaxDim || g_local > RD_MAX_GROUPS) return RD_ERR_UNSUPPORTED;
  *bytes = static_cast<size_t>(linear_act_bwd_bytes(m, n, g_local));
  return RD_OK;
}

extern "C" rd_status rd_linear_act_bwd(const void* d_out, int32_t out_dtype, const void* pre,
                                       int32_t act, void* d_pre, float* d_bias, int64_t m, int64_t n,
                                       const int32_t* group_sizes, int32_t g_total,
                                       int32_t group_offset, int32_t g_local, const int32_t* limit,
                                       void* workspace, size_t workspace_bytes, int32_t* status,
                                       rd_stream_t stream) {
  rd_status st = check_linear(m, 0, n, group_sizes, g_total, group_offset, g_local, limit, status, act, out_dtype);
  if (st != RD_OK) return st;
  if (m > 0 && n > 0 && (d_out == nullptr || (pre == nullptr) != (act == RD_ACT_NONE))) return RD_ERR_INVALID_ARG;
  const uint64_t need = static_cast<uint64_t>(linear_act_bwd_bytes(m, n, g_local));
  if (d_bias != nullptr && n > 0 && need > 0 && workspace == nullptr) return RD_ERR_INVALID_ARG;
  if (!matrix_aligned(d_out, out_dtype) || !aligned16(pre) || !aligned16(d_pre) || !aligned16(d_bias) ||
      !matrix_aligned(workspace, RD_F32))
    return RD_ERR_UNSUPPORTED;
  const uint64_t n2 = static_cast<uint64_t>(m) * static_cast<uint64_t>(n);
  if (any_overlap<3, 5>({{d_pre, n2 * 2},
                         {d_bias, static_cast<uint64_t>(g_local) * static_cast<uint64_t>(n) * 4},
                         {d_bias != nullptr ? workspace : nullptr, workspace_bytes}},
                        {{d_out, n2 * size_of(out_dtype)},
                         {pre, n2 * 2},
                         {group_sizes, static_cast<uint64_t>(g_total) * 4},
                         {limit, 4},
                         {status, 4}}))
    return RD_ERR_INVALID_ARG;
  if (d_bias != nullptr && workspace_bytes < need) return RD_ERR_INVALID_ARG;
  int sms = 0;
  if ((st = current_device(&sms)) != RD_OK) return st;
  if (n == 0 || (m == 0 && d_bias == nullptr) || (d_pre == nullptr && d_bias == nullptr)) return RD_OK;
  ActBwdArgs a = {};
  a.d_out = d_out;
  a.pre = pre;
  a.d_pre = d_pre;
  a.d_bias = d_bias;
  a.parts = static_cast<float*>(workspace);
  a.group_sizes = group_sizes;
  a.limit = limit;
  a.status = status;
  a.m = static_cast<int32_t>(m);
  a.n = static_cast<int32_t>(n);
  a.g_total = g_total;
  a.group_offset = group_offset;
  a.g_local = g_local;
  a.act = act;
  return done(launch_linear_act_bwd(a, out_dtype, sms, cu(stream)));
}
