// layer_norm.cu -- layer norm of rows and its gradients (rd_layer_norm_fwd, rd_layer_norm_bwd).
//
// Both directions are one pass over HBM.  T threads hold a row in registers, V vectors of eight elements each,
// so the mean, the squares about it and the result come from one read; the next row's loads are issued before
// this row's sums, which hides their latency.  Blocks stay on the SM and take rows in turn, so a thread
// keeps the same columns: weight and bias stay in registers, and the backward pass adds its columns'
// d_out * y and d_out there.  At the end each block writes its two sums a column to the workspace and a second
// kernel adds the blocks' sums in their order (no atomics).
#include <cuda_runtime.h>
#include <stdint.h>

#include "block_args.h"
#include "launch.h"
#include "rows.cuh"

namespace rd {
namespace {

// two sums across a row's threads with one barrier (the slots as in row_sum)
template <int T>
__device__ __forceinline__ void row_sum2(float& p, float& q, float2* slot) {
  p = warp_sum(p);
  q = warp_sum(q);
  if (T == 32) return;
  if ((threadIdx.x & 31) == 0) slot[threadIdx.x >> 5] = make_float2(p, q);
  __syncthreads();
  p = q = 0.0f;
#pragma unroll
  for (int i = 0; i < T / 32; ++i) {
    p += slot[i].x;
    q += slot[i].y;
  }
}

// ------------------------------------------------------------------ forward
template <class X, class O, int T, int V>
__global__ void __launch_bounds__(T == 32 ? 256 : T) layer_norm_fwd_kernel(const NormArgs a) {
  constexpr int kRows = T == 32 ? 8 : 1;       // rows of a block at a time
  constexpr bool kHold = V <= 2 && T <= 512;   // weight and bias in registers
  constexpr bool kAhead = V <= 2;              // the next row's loads in flight
  __shared__ float sums[32];
  __shared__ float2 pairs[32];
  pdl_trigger();
  pdl_wait();
  const int t = threadIdx.x % T;
  const int vecs = a.hidden >> 3;
  const int64_t hidden = a.hidden;
  const int32_t L = rows_within(a.limit, a.rows);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
  const float inv = 1.0f / static_cast<float>(a.hidden);
  const X* x = static_cast<const X*>(a.x);
  O* out = static_cast<O*>(a.out);
  int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / T;
  if (row >= L) return;
  Raw8<X> raw[V];
  auto fetch = [&](int64_t r) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (t + i * T < vecs) load_raw(raw[i], x + r * hidden + 8 * (t + i * T));
  };
  auto param = [&](const float* p, int i, float none, float (&v)[8]) {
    if (p != nullptr) {
      load8_param(p + 8 * (t + i * T), v);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = none;
    }
  };
  fetch(row);
  float w[kHold ? V : 1][8], b[kHold ? V : 1][8];
  if (kHold) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (t + i * T < vecs) {
        param(a.weight, i, 1.0f, w[i]);
        param(a.bias, i, 0.0f, b[i]);
      }
  }
  for (; row < L; row += step) {
    float v[V][8];
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (t + i * T < vecs) {
        widen(raw[i], v[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e) s += v[i][e];
      }
    if (kAhead && row + step < L) fetch(row + step);
    const float mean = row_sum<T>(s, sums) * inv;
    // What is left of the mean after its rounding (c) is taken out too: a row far from zero would
    // otherwise be off by an ulp of its mean.
    float c = 0.0f, q = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (t + i * T < vecs) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          v[i][e] -= mean;
          c += v[i][e];
          q = fmaf(v[i][e], v[i][e], q);
        }
      }
    row_sum2<T>(c, q, pairs);
    c *= inv;
    const float var = fmaf(-c, c, q * inv);  // never below zero but by rounding; NaN stays NaN
    const float rstd = 1.0f / sqrtf((var < 0.0f ? 0.0f : var) + a.eps);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (t + i * T < vecs) {
        if (!kHold) {
          param(a.weight, i, 1.0f, w[0]);
          param(a.bias, i, 0.0f, b[0]);
        }
        const float(&wi)[8] = w[kHold ? i : 0];
        const float(&bi)[8] = b[kHold ? i : 0];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] = fmaf((v[i][e] - c) * rstd, wi[e], bi[e]);
        store8(out + row * hidden + 8 * (t + i * T), v[i]);
      }
    if (t == 0 && a.mean != nullptr) {
      a.mean[row] = mean + c;
      a.rstd[row] = rstd;
    }
    if (!kAhead && row + step < L) fetch(row + step);
  }
}

// rows too long for registers: three reads of the row, of which the last two come from L2
template <class X, class O>
__global__ void __launch_bounds__(1024) layer_norm_fwd_long_kernel(const NormArgs a) {
  __shared__ float sums[32];
  __shared__ float2 pairs[32];
  pdl_trigger();
  pdl_wait();
  const int vecs = a.hidden >> 3;
  const int64_t hidden = a.hidden;
  const int32_t L = rows_within(a.limit, a.rows);
  const float inv = 1.0f / static_cast<float>(a.hidden);
  for (int64_t row = blockIdx.x; row < L; row += gridDim.x) {
    const X* x = static_cast<const X*>(a.x) + row * hidden;
    O* out = static_cast<O*>(a.out) + row * hidden;
    float s = 0.0f, c = 0.0f, q = 0.0f;
    for (int64_t v = threadIdx.x; v < vecs; v += 1024) {
      float e[8];
      load8(x + 8 * v, e);
      s += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
    }
    const float mean = row_sum<1024>(s, sums) * inv;
    for (int64_t v = threadIdx.x; v < vecs; v += 1024) {
      float e[8];
      load8(x + 8 * v, e);
      float k = 0.0f, p = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        k += e[i] - mean;
        p = fmaf(e[i] - mean, e[i] - mean, p);
      }
      c += k;
      q += p;
    }
    row_sum2<1024>(c, q, pairs);
    c *= inv;
    const float var = fmaf(-c, c, q * inv);  // never below zero but by rounding; NaN stays NaN
    const float rstd = 1.0f / sqrtf((var < 0.0f ? 0.0f : var) + a.eps);
    for (int64_t v = threadIdx.x; v < vecs; v += 1024) {
      float e[8], w[8], b[8];
      load8(x + 8 * v, e);
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = 1.0f, b[i] = 0.0f;
      if (a.weight != nullptr) load8_param(a.weight + 8 * v, w);
      if (a.bias != nullptr) load8_param(a.bias + 8 * v, b);
#pragma unroll
      for (int i = 0; i < 8; ++i) e[i] = fmaf((e[i] - mean - c) * rstd, w[i], b[i]);
      store8(out + 8 * v, e);
    }
    if (threadIdx.x == 0 && a.mean != nullptr) {
      a.mean[row] = mean + c;
      a.rstd[row] = rstd;
    }
  }
}

// ------------------------------------------------------------------ backward
template <class X, class O, int T, int V>
__global__ void __launch_bounds__(T == 32 ? 256 : T) layer_norm_bwd_kernel(const NormArgs a) {
  constexpr int kRows = T == 32 ? 8 : 1;
  __shared__ float2 slots[2][32];
  __shared__ float across[T == 32 ? kRows * 2 * 256 : 1];
  pdl_trigger();
  pdl_wait();
  const int t = threadIdx.x % T;
  const int vecs = a.hidden >> 3;
  const int64_t hidden = a.hidden;
  const int32_t L = rows_within(a.limit, a.rows);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
  const float inv = 1.0f / static_cast<float>(a.hidden);
  const X* x = static_cast<const X*>(a.x);
  const O* d_out = static_cast<const O*>(a.d_out);
  X* d_x = static_cast<X*>(a.out);
  int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / T;
  Raw8<X> rx[V];
  Raw8<O> rd_[V];
  float mean_next = 0.0f, rstd_next = 0.0f;
  auto fetch = [&](int64_t r) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (t + i * T < vecs) {
        load_raw(rx[i], x + r * hidden + 8 * (t + i * T));
        load_raw(rd_[i], d_out + r * hidden + 8 * (t + i * T));
      }
    mean_next = a.mean[r];
    rstd_next = a.rstd[r];
  };
  if (row < L) fetch(row);
  float w[V][8], dw[V][8], db[V][8];
#pragma unroll
  for (int i = 0; i < V; ++i) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      w[i][e] = 1.0f;
      dw[i][e] = db[i][e] = 0.0f;
    }
    if (a.weight != nullptr && t + i * T < vecs) load8_param(a.weight + 8 * (t + i * T), w[i]);
  }
  int slot = 0;
  for (; row < L; row += step) {
    float y[V][8], d[V][8];
    const float mean = mean_next, rstd = rstd_next;
    float p = 0.0f, q = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (t + i * T < vecs) {
        widen(rx[i], y[i]);
        widen(rd_[i], d[i]);
      }
    if (row + step < L) fetch(row + step);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (t + i * T < vecs) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          y[i][e] = (y[i][e] - mean) * rstd;
          dw[i][e] = fmaf(d[i][e], y[i][e], dw[i][e]);
          db[i][e] += d[i][e];
          d[i][e] *= w[i][e];
          p += d[i][e];
          q = fmaf(d[i][e], y[i][e], q);
        }
      }
    row_sum2<T>(p, q, slots[slot]);
    slot ^= 1;
    p *= inv;
    q *= inv;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (t + i * T < vecs) {
#pragma unroll
        for (int e = 0; e < 8; ++e) d[i][e] = rstd * (d[i][e] - fmaf(y[i][e], q, p));
        store8(d_x + row * hidden + 8 * (t + i * T), d[i]);
      }
  }
  if (a.parts == nullptr) return;
  float* part = a.parts + static_cast<int64_t>(blockIdx.x) * 2 * hidden;
  if (T == 32) {
    // the block's warps hold the same columns: added in their order through shared memory
    const int warp = threadIdx.x >> 5;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      across[(warp * 2) * 256 + t * 8 + e] = dw[0][e];
      across[(warp * 2 + 1) * 256 + t * 8 + e] = db[0][e];
    }
    __syncthreads();
    for (int c = threadIdx.x; c < 512; c += 256) {
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < kRows; ++i) s += across[i * 512 + c];
      const int col = c & 255;
      if (col < hidden) part[(c >> 8) * hidden + col] = s;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (t + i * T < vecs) {
      store8(part + 8 * (t + i * T), dw[i]);
      store8(part + hidden + 8 * (t + i * T), db[i]);
    }
}

// rows too long for registers: d_x alone, the row read twice (the second time from L2)
template <class X, class O>
__global__ void __launch_bounds__(1024) layer_norm_dx_long_kernel(const NormArgs a) {
  __shared__ float2 slots[2][32];
  pdl_trigger();
  pdl_wait();
  const int vecs = a.hidden >> 3;
  const int64_t hidden = a.hidden;
  const int32_t L = rows_within(a.limit, a.rows);
  const float inv = 1.0f / static_cast<float>(a.hidden);
  int slot = 0;
  for (int64_t row = blockIdx.x; row < L; row += gridDim.x, slot ^= 1) {
    const X* x = static_cast<const X*>(a.x) + row * hidden;
    const O* d_out = static_cast<const O*>(a.d_out) + row * hidden;
    X* d_x = static_cast<X*>(a.out) + row * hidden;
    const float mean = a.mean[row], rstd = a.rstd[row];
    float p = 0.0f, q = 0.0f;
    auto at = [&](int64_t v, float (&y)[8], float (&d)[8]) {
      load8(x + 8 * v, y);
      load8(d_out + 8 * v, d);
      if (a.weight != nullptr) {
        float w[8];
        load8_param(a.weight + 8 * v, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] *= w[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = (y[i] - mean) * rstd;
    };
    for (int64_t v = threadIdx.x; v < vecs; v += 1024) {
      float y[8], d[8], pv = 0.0f, qv = 0.0f;
      at(v, y, d);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        pv += d[i];
        qv = fmaf(d[i], y[i], qv);
      }
      p += pv;
      q += qv;
    }
    row_sum2<1024>(p, q, slots[slot]);
    p *= inv;
    q *= inv;
    for (int64_t v = threadIdx.x; v < vecs; v += 1024) {
      float y[8], d[8];
      at(v, y, d);
#pragma unroll
      for (int i = 0; i < 8; ++i) d[i] = rstd * (d[i] - fmaf(y[i], q, p));
      store8(d_x + 8 * v, d);
    }
  }
}

// ... and their columns' sums over a chunk of rows: 256 columns a block, eight rows at a time
template <class X, class O>
__global__ void __launch_bounds__(256) layer_norm_columns_kernel(const NormArgs a, int32_t chunk_rows) {
  __shared__ float across[8][2][256];
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t hidden = a.hidden;
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 256 + lane * 8;
  const int32_t L = rows_within(a.limit, a.rows);
  const int64_t lo = static_cast<int64_t>(blockIdx.y) * chunk_rows;
  const int64_t hi = lo + chunk_rows < L ? lo + chunk_rows : L;
  float dw[8], db[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) dw[i] = db[i] = 0.0f;
  if (col < hidden) {
#pragma unroll 4
    for (int64_t row = lo + warp; row < hi; row += 8) {
      float y[8], d[8];
      load8(static_cast<const X*>(a.x) + row * hidden + col, y);
      load8(static_cast<const O*>(a.d_out) + row * hidden + col, d);
      const float mean = a.mean[row], rstd = a.rstd[row];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        dw[i] = fmaf(d[i], (y[i] - mean) * rstd, dw[i]);
        db[i] += d[i];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    across[warp][0][lane * 8 + i] = dw[i];
    across[warp][1][lane * 8 + i] = db[i];
  }
  __syncthreads();
  float* part = a.parts + static_cast<int64_t>(blockIdx.y) * 2 * hidden;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (c >= hidden) return;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += across[i][k][threadIdx.x];
    part[k * hidden + c] = s;
  }
}

// The blocks' sums to the gradients: 32 columns a block, eight threads a column, each every eighth
// part in order.
__global__ void __launch_bounds__(256) layer_norm_parts_kernel(const NormArgs a, int32_t parts) {
  __shared__ float across[8][33];
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t cols = 2 * static_cast<int64_t>(a.hidden);
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float s = 0.0f;
  if (c < cols) {
    const float* p = a.parts + c;
#pragma unroll 8
    for (int i = warp; i < parts; i += 8) s += p[i * cols];
  }
  across[warp][lane] = s;
  __syncthreads();
  if (warp != 0 || c >= cols) return;
  s = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s += across[i][lane];
  float* out = c < a.hidden ? a.d_weight : a.d_bias;
  if (out != nullptr) out[c < a.hidden ? c : c - a.hidden] = s;
}

int64_t ceil_of(int64_t n, int64_t d) { return (n + d - 1) / d; }

template <class X, class O, int T, int V>
cudaError_t fwd(const NormArgs& a, int sms, cudaStream_t stream) {
  constexpr int kRows = T == 32 ? 8 : 1, threads = T == 32 ? 256 : T;
  const int64_t blocks = ceil_of(a.rows, kRows), most = static_cast<int64_t>(sms) * (T >= 1024 ? 1 : 1024 / threads);
  return launch_pdl(layer_norm_fwd_kernel<X, O, T, V>, dim3(static_cast<unsigned>(blocks < most ? blocks : most)),
                    threads, 0, 1, stream, a);
}

template <class X, class O>
cudaError_t fwd_by_width(const NormArgs& a, int sms, cudaStream_t stream) {
  const int vecs = a.hidden / 8;
  if (vecs <= 32) return fwd<X, O, 32, 1>(a, sms, stream);
  if (vecs <= 64) return fwd<X, O, 32, 2>(a, sms, stream);
  if (vecs <= 128) return fwd<X, O, 128, 1>(a, sms, stream);
  if (vecs <= 256) return fwd<X, O, 128, 2>(a, sms, stream);
  if (vecs <= 512) return fwd<X, O, 256, 2>(a, sms, stream);
  if (vecs <= 1024) return fwd<X, O, 512, 2>(a, sms, stream);
  if (vecs <= 2048) return fwd<X, O, 1024, 2>(a, sms, stream);
  if (vecs <= 4096) return fwd<X, O, 1024, 4>(a, sms, stream);
  const int64_t most = 2 * static_cast<int64_t>(sms);
  return launch_pdl(layer_norm_fwd_long_kernel<X, O>, dim3(static_cast<unsigned>(a.rows < most ? a.rows : most)),
                    1024, 0, 1, stream, a);
}

// threads of a row of the backward kernel that holds rows in registers; 0: rows are too long for it
int bwd_threads(int64_t hidden) {
  const int64_t vecs = hidden / 8;
  return vecs <= 32 ? 32 : (vecs <= 128 ? 128 : (vecs <= 256 ? 256 : (vecs <= 1024 ? 512 : 0)));
}

template <class X, class O, int T, int V>
cudaError_t bwd(const NormArgs& a, int parts, cudaStream_t stream) {
  return launch_pdl(layer_norm_bwd_kernel<X, O, T, V>, dim3(static_cast<unsigned>(parts)), T == 32 ? 256 : T, 0, 1,
                    stream, a);
}

template <class X, class O>
cudaError_t bwd_by_width(const NormArgs& a, int parts, int sms, cudaStream_t stream) {
  const int vecs = a.hidden / 8;
  switch (bwd_threads(a.hidden)) {
    case 32: return bwd<X, O, 32, 1>(a, parts, stream);
    case 128: return bwd<X, O, 128, 1>(a, parts, stream);
    case 256: return bwd<X, O, 256, 1>(a, parts, stream);
    case 512: return vecs <= 512 ? bwd<X, O, 512, 1>(a, parts, stream) : bwd<X, O, 512, 2>(a, parts, stream);
    default: break;
  }
  const int64_t most = 2 * static_cast<int64_t>(sms);
  if (a.rows > 0) {
    const cudaError_t e = launch_pdl(layer_norm_dx_long_kernel<X, O>,
                                     dim3(static_cast<unsigned>(a.rows < most ? a.rows : most)), 1024, 0, 1, stream, a);
    if (e != cudaSuccess) return e;
  }
  if (a.parts == nullptr) return cudaSuccess;
  return launch_pdl(layer_norm_columns_kernel<X, O>,
                    dim3(static_cast<unsigned>(ceil_of(a.hidden, 256)), static_cast<unsigned>(parts)), 256, 0, 1,
                    stream, a, static_cast<int32_t>(ceil_of(a.rows, parts)));
}

}  // namespace

cudaError_t launch_layer_norm_fwd(const NormArgs& a, int dtype, int out_dtype, int sms,
                                  cudaStream_t stream) {
  if (dtype == RD_F32)
    return out_dtype == RD_F32 ? fwd_by_width<float, float>(a, sms, stream)
                               : fwd_by_width<float, bf16>(a, sms, stream);
  return out_dtype == RD_F32 ? fwd_by_width<bf16, float>(a, sms, stream)
                             : fwd_by_width<bf16, bf16>(a, sms, stream);
}

int layer_norm_bwd_parts(int64_t rows, int64_t hidden, int sms) {
  const int threads = bwd_threads(hidden);
  if (threads == 0) {
    const int64_t p = ceil_of(rows, 64);
    return static_cast<int>(p < 1 ? 1 : (p < 64 ? p : 64));
  }
  const int64_t per_block = threads == 32 ? 8 : 1;
  const int64_t p = ceil_of(rows, 4 * per_block), most = static_cast<int64_t>(sms) * (threads == 32 ? 4 : 1024 / threads);
  return static_cast<int>(p < 1 ? 1 : (p < most ? p : most));
}

cudaError_t launch_layer_norm_bwd(const NormArgs& a, int dtype, int out_dtype, int sms,
                                  cudaStream_t stream) {
  const int parts = layer_norm_bwd_parts(a.rows, a.hidden, sms);
  cudaError_t e;
  if (dtype == RD_F32)
    e = out_dtype == RD_F32 ? bwd_by_width<float, float>(a, parts, sms, stream)
                            : bwd_by_width<float, bf16>(a, parts, sms, stream);
  else
    e = out_dtype == RD_F32 ? bwd_by_width<bf16, float>(a, parts, sms, stream)
                            : bwd_by_width<bf16, bf16>(a, parts, sms, stream);
  if (e != cudaSuccess || a.parts == nullptr) return e;
  return launch_pdl(layer_norm_parts_kernel, dim3(static_cast<unsigned>(ceil_of(2 * static_cast<int64_t>(a.hidden), 32))),
                    256, 0, 1, stream, a, static_cast<int32_t>(parts));
}

}  // namespace rd
