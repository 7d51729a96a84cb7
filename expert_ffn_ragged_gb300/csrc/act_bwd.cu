// act_bwd.cu -- the gradients of rd_linear in front of its activation (rd_linear_act_bwd).
//
// One pass: d_out and pre are read once, d_pre is written once, and the column sums of the unrounded
// products, group by group, come from the same registers.  The rows of a group are cut into chunks; a block
// takes a chunk and W vectors of columns, 256 / W rows at a time, adds its rows' products in registers
// and across its threads in a fixed order, and writes one sum a column to the workspace; a second
// kernel adds a group's chunks in their order (no atomics).  Where all rows are few, a whole group is one chunk and its
// sums are the result: one launch, no workspace.
#include <cuda_runtime.h>
#include <stdint.h>

#include "act_math.cuh"
#include "block_args.h"
#include "gemm_args.h"
#include "launch.h"
#include "rows.cuh"

namespace rd {
namespace {

constexpr int kActThreads = 256;
constexpr int kActBatch = 4;                  // rows of a thread in flight
constexpr int kActBlocks = 3;                 // blocks on an SM
constexpr int32_t kChunkRows = 64;            // fewest rows of a chunk that is not a whole group
constexpr int32_t kWholeGroups = 0;           // chunk_rows: every group is one chunk
constexpr int64_t kPartsAt = 4 * (kMaxGroups + 4);  // bytes of the workspace before the sums

struct Chunks {
  int32_t bound[kMaxGroups + 1];  // group boundaries, clamped to L
  int32_t start[kMaxGroups + 1];  // first chunk of each local group
  int32_t L;
  int32_t zero_lo, zero_hi;       // rows [0, zero_lo) and [zero_hi, L) of d_pre are zero
  int32_t zeros_lo, zeros;        // chunks of the first range, and of both
};

// Run by one warp; the sums of group sizes in 64 bits.
__device__ __forceinline__ void build_chunks(Chunks& sh, const ActBwdArgs& a, int lane) {
  const int32_t L = rows_within(a.limit, a.m);
  auto size_of = [&](int i) { return a.group_sizes != nullptr ? a.group_sizes[i] : a.m; };
  auto scan = [&](long long v) {
    long long incl = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long o = __shfl_up_sync(0xFFFFFFFFu, incl, d);
      if (lane >= d) incl += o;
    }
    return incl - v;
  };
  const int G = a.g_total, per = (G + 31) / 32, lo = min(lane * per, G), hi = min(lo + per, G);
  long long sum = 0;
  bool neg = false;
  for (int i = lo; i < hi; ++i) {
    const int32_t s = size_of(i);
    neg |= s < 0;
    sum += s > 0 ? s : 0;
  }
  long long run = scan(sum);
  for (int i = lo; i < hi; ++i) {
    sh.bound[i] = clamp_boundary(run, L);
    const int32_t s = size_of(i);
    run += s > 0 ? s : 0;
  }
  const long long total = __shfl_sync(0xFFFFFFFFu, run, 31);
  neg = __any_sync(0xFFFFFFFFu, neg);
  if (lane == 0) {
    sh.bound[G] = clamp_boundary(total, L);
    sh.L = L;
    if (a.status != nullptr && blockIdx.x == 0) {
      const int bits = (neg ? RD_STATUS_NEG_SIZE : 0) | (total > a.m ? RD_STATUS_OVERFLOW : 0);
      if (bits) atomicOr(a.status, bits);
    }
  }
  __syncwarp();
  const int32_t R = a.chunk_rows;
  auto chunks_of = [&](int j) -> long long {
    if (R == kWholeGroups) return 1;
    return ceil_div(sh.bound[a.group_offset + j + 1] - sh.bound[a.group_offset + j], R);
  };
  const int GL = a.g_local, per2 = (GL + 31) / 32, lo2 = min(lane * per2, GL), hi2 = min(lo2 + per2, GL);
  long long mine = 0;
  for (int j = lo2; j < hi2; ++j) mine += chunks_of(j);
  long long at = scan(mine);
  for (int j = lo2; j < hi2; ++j) {
    sh.start[j] = static_cast<int32_t>(at);
    at += chunks_of(j);
  }
  at = __shfl_sync(0xFFFFFFFFu, at, 31);
  if (lane == 0) {
    sh.start[GL] = static_cast<int32_t>(at);
    sh.zero_lo = sh.bound[a.group_offset];
    sh.zero_hi = sh.bound[a.group_offset + GL];
    const int32_t zr = kChunkRows;
    sh.zeros_lo = a.d_pre != nullptr ? ceil_div(sh.zero_lo, zr) : 0;
    sh.zeros = sh.zeros_lo + (a.d_pre != nullptr ? ceil_div(L - sh.zero_hi, zr) : 0);
  }
}

template <class D, int ACT, int W>
__device__ __forceinline__ void act_bwd_chunk(const ActBwdArgs& a, int32_t lo, int32_t hi, int64_t col,
                                              bool on, int row_lane, float2 (&sum)[4]) {
  constexpr int kLanes = kActThreads / W;
  const D* d_out = static_cast<const D*>(a.d_out);
  const bf16* pre = static_cast<const bf16*>(a.pre);
  bf16* d_pre = static_cast<bf16*>(a.d_pre);
  const int64_t n = a.n;
  if (!on) return;
  const int64_t step = static_cast<int64_t>(kLanes) * n;
  int64_t at = (static_cast<int64_t>(lo) + row_lane) * n + col;
  for (int32_t left = hi - lo - row_lane; left > 0; left -= kLanes * kActBatch, at += step * kActBatch) {
    Raw8<D> rd_[kActBatch];
    Raw8<bf16> rp[kActBatch];
#pragma unroll
    for (int b = 0; b < kActBatch; ++b) {
      if (left > b * kLanes) {
        load_raw(rd_[b], d_out + at + b * step);
        if (ACT != RD_ACT_NONE) load_raw(rp[b], pre + at + b * step);
      }
    }
#pragma unroll
    for (int b = 0; b < kActBatch; ++b) {
      if (left > b * kLanes) {
        float d[8];
        widen(rd_[b], d);
        if (ACT != RD_ACT_NONE) {
          float z[8];
          widen(rp[b], z);
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            const float2 r = mul2(make_float2(d[e], d[e + 1]), act_slope<ACT>(make_float2(z[e], z[e + 1])));
            d[e] = r.x;
            d[e + 1] = r.y;
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[e] = add2(sum[e], make_float2(d[2 * e], d[2 * e + 1]));
        if (d_pre != nullptr) store8(d_pre + at + b * step, d);
      }
    }
  }
}

// W: vectors of columns of a block
template <class D, int ACT, int W>
__global__ void __launch_bounds__(kActThreads, kActBlocks) linear_act_bwd_kernel(const ActBwdArgs a) {
  constexpr int kLanes = kActThreads / W;
  __shared__ Chunks sh;
  __shared__ __align__(16) float across[kLanes][W * 8];  // pairs are stored at once
  pdl_trigger();
  pdl_wait();
  if (threadIdx.x < 32) build_chunks(sh, a, threadIdx.x);
  __syncthreads();
  const int col_lane = threadIdx.x % W, row_lane = threadIdx.x / W;
  const int64_t n = a.n;
  const int64_t col_blocks = (n + W * 8 - 1) / (W * 8);
  const int32_t chunks = sh.start[a.g_local];
  const int64_t units = (static_cast<int64_t>(chunks) + sh.zeros) * col_blocks;
  const bool whole = a.chunk_rows == kWholeGroups;
  if (!whole && blockIdx.x == 0 && a.d_bias != nullptr) {
    // the second kernel finds a group's chunks here
    int32_t* head = reinterpret_cast<int32_t*>(a.parts);
    for (int j = threadIdx.x; j <= a.g_local; j += kActThreads) head[j] = sh.start[j];
  }
  float* parts = whole ? a.d_bias : a.parts + kPartsAt / 4;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int32_t chunk = static_cast<int32_t>(u / col_blocks);
    const int64_t col0 = (u - chunk * col_blocks) * (W * 8), col = col0 + col_lane * 8;
    const bool on = col < n;
    if (chunk >= chunks) {
      const int32_t z = chunk - chunks;
      const bool low = z < sh.zeros_lo;
      const int32_t lo = low ? z * kChunkRows : sh.zero_hi + (z - sh.zeros_lo) * kChunkRows;
      const int32_t end = low ? sh.zero_lo : sh.L;
      const int32_t hi = end - lo > kChunkRows ? lo + kChunkRows : end;
      if (on)
        for (int32_t r = lo + row_lane; r < hi; r += kLanes)
          *reinterpret_cast<uint4*>(static_cast<bf16*>(a.d_pre) + r * n + col) = make_uint4(0, 0, 0, 0);
      continue;
    }
    int j = 0, top = a.g_local;  // the last group that starts at or before the chunk: it has rows (or is whole)
    if (whole) j = top = chunk;
    while (top - j > 1) {
      const int mid = (j + top) >> 1;
      if (sh.start[mid] <= chunk) j = mid; else top = mid;
    }
    const int32_t re = sh.bound[a.group_offset + j + 1];
    int32_t lo = sh.bound[a.group_offset + j], hi = re;
    if (!whole) {
      lo += (chunk - sh.start[j]) * a.chunk_rows;
      hi = re - lo > a.chunk_rows ? lo + a.chunk_rows : re;
    }
    float2 sum[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[e] = both(0.0f);
    act_bwd_chunk<D, ACT, W>(a, lo, hi, col, on, row_lane, sum);
    if (a.d_bias == nullptr) continue;
    __syncthreads();  // the sums of the unit before have been read
#pragma unroll
    for (int e = 0; e < 4; ++e)
      *reinterpret_cast<float2*>(&across[row_lane][col_lane * 8 + 2 * e]) = sum[e];
    __syncthreads();
    for (int c = threadIdx.x; c < W * 8; c += kActThreads) {
      if (col0 + c >= n) continue;
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < kLanes; ++i) s += across[i][c];
      parts[(whole ? j : chunk) * n + col0 + c] = s;
    }
  }
}

// A group's chunks to its gradient: 128 columns a block, eight warps that each take every eighth chunk in
// order.
__global__ void __launch_bounds__(256) linear_bias_parts_kernel(const ActBwdArgs a) {
  __shared__ float4 across[8][32];
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t n = a.n, col_blocks = (n + 127) / 128;
  const int32_t* head = reinterpret_cast<const int32_t*>(a.parts);
  const float* parts = a.parts + kPartsAt / 4;
  const int64_t units = col_blocks * a.g_local;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int64_t j = u / col_blocks, col = (u - j * col_blocks) * 128 + lane * 4;
    const int32_t lo = head[j], hi = head[j + 1];
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (col < n) {
#pragma unroll 8
      for (int32_t c = lo + warp; c < hi; c += 8) {
        const float4 p = *reinterpret_cast<const float4*>(parts + c * n + col);
        s.x += p.x;
        s.y += p.y;
        s.z += p.z;
        s.w += p.w;
      }
    }
    __syncthreads();
    across[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && col < n) {
      s = across[0][lane];
#pragma unroll
      for (int i = 1; i < 8; ++i) {
        const float4 p = across[i][lane];
        s.x += p.x;
        s.y += p.y;
        s.z += p.z;
        s.w += p.w;
      }
      *reinterpret_cast<float4*>(a.d_bias + j * n + col) = s;
    }
  }
}

template <class D, int ACT, int W>
cudaError_t go(ActBwdArgs a, int64_t chunks, int sms, cudaStream_t stream) {
  const int64_t units = chunks * ((static_cast<int64_t>(a.n) + W * 8 - 1) / (W * 8));
  const int64_t most = static_cast<int64_t>(sms) * kActBlocks;
  return launch_pdl(linear_act_bwd_kernel<D, ACT, W>, dim3(static_cast<unsigned>(units < most ? units : most)), kActThreads,
                    0, 1, stream, a);
}

template <class D, int ACT>
cudaError_t by_width(ActBwdArgs a, int sms, cudaStream_t stream) {
  // Whole groups where no more than 2048 rows could meet in one group; chunks of 256 rows where they
  // still leave each SM eight blocks' work, else of 64.
  const bool whole = a.m <= 2048;
  a.chunk_rows = whole ? kWholeGroups
                       : (static_cast<int64_t>(a.m) / 256 * ((a.n + 255) / 256) >= 8 * static_cast<int64_t>(sms)
                              ? 4 * kChunkRows
                              : kChunkRows);
  const int64_t chunks = whole ? a.g_local + (a.m + kChunkRows - 1) / kChunkRows
                               : static_cast<int64_t>(a.m) / a.chunk_rows + 1 + a.g_local;
  cudaError_t e;
  if (whole || a.n <= 64) e = go<D, ACT, 8>(a, chunks, sms, stream);
  else if (a.n <= 128) e = go<D, ACT, 16>(a, chunks, sms, stream);
  else e = go<D, ACT, 32>(a, chunks, sms, stream);
  if (e != cudaSuccess || whole || a.d_bias == nullptr) return e;
  const int64_t units = (static_cast<int64_t>(a.n) + 127) / 128 * a.g_local, most = static_cast<int64_t>(sms) * 8;
  return launch_pdl(linear_bias_parts_kernel, dim3(static_cast<unsigned>(units < most ? units : most)), 256, 0, 1,
                    stream, a);
}

}  // namespace

int64_t linear_act_bwd_bytes(int64_t m, int64_t n, int32_t g_local) {
  return kPartsAt + 4 * n * ((m + kChunkRows - 1) / kChunkRows + g_local);
}

namespace {
template <class D>
cudaError_t by_act(const ActBwdArgs& a, int sms, cudaStream_t stream) {
  switch (a.act) {
    case RD_ACT_RELU: return by_width<D, RD_ACT_RELU>(a, sms, stream);
    case RD_ACT_GELU: return by_width<D, RD_ACT_GELU>(a, sms, stream);
    case RD_ACT_GELU_TANH: return by_width<D, RD_ACT_GELU_TANH>(a, sms, stream);
    case RD_ACT_SILU: return by_width<D, RD_ACT_SILU>(a, sms, stream);
    default: return by_width<D, RD_ACT_NONE>(a, sms, stream);
  }
}
}  // namespace

cudaError_t launch_linear_act_bwd(const ActBwdArgs& a, int out_dtype, int sms, cudaStream_t stream) {
  return out_dtype == RD_F32 ? by_act<float>(a, sms, stream) : by_act<bf16>(a, sms, stream);
}

}  // namespace rd
