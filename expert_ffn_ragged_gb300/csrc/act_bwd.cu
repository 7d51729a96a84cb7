// act_bwd.cu -- the gradients of rd_linear in front of its activation (rd_linear_act_bwd).
//
// One pass: d_out and pre are read once, d_pre is written once, and the column sums of the unrounded
// products, group by group, come from the same registers.  A block takes W vectors of eight columns and one of
// P equal shares of the rows, 256 / W rows at a time with the next two on their way to shared memory; P is as many as
// run at once.  It keeps its sums in registers until its rows' group ends, then adds its threads' in a fixed order
// and writes one sum a column to the workspace.  Along the rows p and j only rise, so no two meetings of a
// share p and a group j have the same p + j, and that numbers the sums; a second kernel adds a group's in their
// order (no atomics).  A few rows, or some over many groups, are taken a group a block instead: its sums are the
// result, and there is neither a workspace nor a second launch (2048 x 1024, 64 groups: 8.0 us against 10.1).
//
// Bound: HBM.  16384 x 14336, exact gelu, bf16: 1.41 GB in 227 us (6.2 TB/s), the tanh form 220; issue slots come next (58 % of
// them are taken).
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "act_math.cuh"
#include "block_args.h"
#include "gemm_args.h"
#include "launch.h"
#include "rows.cuh"

namespace rd {
namespace {

constexpr int kActThreads = 256;
constexpr int kActStages = 3;                 // rows of a thread in its ring
// blocks on an SM: with two streams in and one out, three of them have more on their way than is good (16384 x 14336, us
// three / two: gelu 239 / 227, tanh form 239 / 220; without an activation 147 / 166)
template <int ACT>
constexpr int kActBlocks = ACT == RD_ACT_NONE ? 3 : 2;
template <int ACT>
constexpr int kActSlots = 152 * kActBlocks<ACT>;  // blocks that run at once
constexpr int kActMostSlots = kActSlots<RD_ACT_NONE>;
constexpr int kActLeastRows = 16;             // rows of a share
// the workspace before the sums: rows of a share, then the local groups' boundaries
constexpr int64_t kPartsAt = 4 * (kMaxGroups + 8);

struct Bounds {
  int32_t bound[kMaxGroups + 1];  // group boundaries, clamped to L
  int32_t L;
};

// Run by one warp; the sums of group sizes in 64 bits.
__device__ __forceinline__ void build_bounds(Bounds& sh, const ActBwdArgs& a, int lane) {
  const int32_t L = rows_within(a.limit, a.m);
  auto size_of = [&](int i) { return a.group_sizes != nullptr ? a.group_sizes[i] : a.m; };
  const int G = a.g_total, per = (G + 31) / 32, lo = min(lane * per, G), hi = min(lo + per, G);
  long long sum = 0;
  bool neg = false;
  for (int i = lo; i < hi; ++i) {
    const int32_t s = size_of(i);
    neg |= s < 0;
    sum += s > 0 ? s : 0;
  }
  long long incl = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long o = __shfl_up_sync(0xFFFFFFFFu, incl, d);
    if (lane >= d) incl += o;
  }
  long long run = incl - sum;
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
}

// A thread's eight columns of one row, on their way to or in shared memory.  bf16 is one 16-byte copy.  f32
// is two, and so that a warp's copies are whole lines, lane l copies the 16-byte pieces l and l + W of its row's 2 W
// and finds its own, 2 l and 2 l + 1, after the warp's barrier.
template <class D, int W>
struct RowPiece;
template <int W>
struct RowPiece<bf16, W> {
  static constexpr int kBytes = 16;  // of a thread
  static __device__ __forceinline__ void fetch(uint8_t* block, int thread, const bf16* row, int lane, int64_t cols) {
    if (8 * lane < cols)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                       static_cast<uint32_t>(__cvta_generic_to_shared(block + 16 * thread))),
                   "l"(row + 8 * lane)
                   : "memory");
  }
  static __device__ __forceinline__ void read(const uint8_t* block, int thread, float (&v)[8]) {
    const uint4 r = *reinterpret_cast<const uint4*>(block + 16 * thread);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_lo(w[i]);
      v[2 * i + 1] = bf16_hi(w[i]);
    }
  }
};
template <int W>
struct RowPiece<float, W> {
  static constexpr int kBytes = 32;
  static __device__ __forceinline__ void fetch(uint8_t* block, int thread, const float* row, int lane, int64_t cols) {
    uint8_t* to = block + 32 * (thread - lane);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int piece = lane + h * W;
      if (4 * piece < cols) quad_copy(reinterpret_cast<float4*>(to) + piece, row + 4 * piece);
    }
  }
  static __device__ __forceinline__ void read(const uint8_t* block, int thread, float (&v)[8]) {
    const float4* p = reinterpret_cast<const float4*>(block + 32 * thread);
    const float4 x = p[0], y = p[1];
    v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w, v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
  }
};

// Rows [lo, hi), columns [col0, col0 + 8 W): a row a thread at a time, the next kActStages - 1 on their way.
template <class D, int ACT, int W>
__device__ __forceinline__ void act_bwd_rows(const ActBwdArgs& a, int32_t lo, int32_t hi, int64_t col0, uint8_t* ring,
                                              float2 (&sum)[4]) {
  using PD = RowPiece<D, W>;
  using PZ = RowPiece<bf16, W>;
  constexpr int kLanes = kActThreads / W;
  constexpr int kStage = kActThreads * (PD::kBytes + (ACT != RD_ACT_NONE ? PZ::kBytes : 0));
  const int lane = threadIdx.x % W;
  const int64_t n = a.n, cols = n - col0;
  const int row_lane = threadIdx.x / W;
  const int32_t left = hi - lo - row_lane;  // rows from this thread's first one on
  const int64_t step = static_cast<int64_t>(kLanes) * n;
  const int64_t at = (static_cast<int64_t>(lo) + row_lane) * n + col0;  // of this thread's first row
  const D* d_out = static_cast<const D*>(a.d_out);
  const bf16* pre = static_cast<const bf16*>(a.pre);
  bf16* d_pre = static_cast<bf16*>(a.d_pre);
  const bool on = 8 * lane < cols;
  // every thread of a warp takes as many turns as its first row lane (32 / W rows a warp)
  const int32_t warp_left = hi - lo - static_cast<int32_t>(threadIdx.x & ~31u) / W;
  const int turns = warp_left > 0 ? (warp_left - 1) / kLanes + 1 : 0;
  auto fetch = [&](int turn, int stage) {
    if (turn * kLanes < left) {
      uint8_t* to = ring + stage * kStage;
      PD::fetch(to, threadIdx.x, d_out + at + turn * step, lane, cols);
      if (ACT != RD_ACT_NONE)
        PZ::fetch(to + kActThreads * PD::kBytes, threadIdx.x, pre + at + turn * step, lane, cols);
    }
    copies_commit();
  };
#pragma unroll
  for (int s = 0; s < kActStages - 1; ++s) fetch(s, s);
  int stage = 0;
#pragma unroll 1
  for (int turn = 0; turn < turns; ++turn) {
    if (PD::kBytes == 32) __syncwarp();  // the stage's pieces have been read
    fetch(turn + kActStages - 1, stage == 0 ? kActStages - 1 : stage - 1);
    copies_wait<kActStages - 1>();
    if (PD::kBytes == 32) __syncwarp();  // the other lanes' pieces are there too
    if (on && turn * kLanes < left) {
      const uint8_t* from = ring + stage * kStage;
      float d[8];
      PD::read(from, threadIdx.x, d);
      if (ACT != RD_ACT_NONE) {
        float z[8];
        PZ::read(from + kActThreads * PD::kBytes, threadIdx.x, z);
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const float2 r = mul2(make_float2(d[e], d[e + 1]), act_slope<ACT>(make_float2(z[e], z[e + 1])));
          d[e] = r.x;
          d[e + 1] = r.y;
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[e] = add2(sum[e], make_float2(d[2 * e], d[2 * e + 1]));
      if (d_pre != nullptr) store8(d_pre + at + turn * step + 8 * lane, d);
    }
    if (++stage == kActStages) stage = 0;
  }
  copies_wait<0>();
  if (PD::kBytes == 32) __syncwarp();
}

// W: vectors of columns of a block
template <class D, int ACT, int W>
__global__ void __launch_bounds__(kActThreads, kActBlocks<ACT>) linear_act_bwd_kernel(const ActBwdArgs a) {
  constexpr int kLanes = kActThreads / W;
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ Bounds sh;
  __shared__ __align__(16) float across[kLanes][W * 8];  // pairs are stored at once
  pdl_trigger();
  pdl_wait();
  if (threadIdx.x < 32) build_bounds(sh, a, threadIdx.x);
  __syncthreads();
  const int col_lane = threadIdx.x % W, row_lane = threadIdx.x / W;
  const int64_t n = a.n;
  const int32_t col_blocks = ceil_div(a.n, W * 8);
  const int32_t L = sh.L, rows = max(ceil_div(L, max(a.shares, 1)), 1);
  const int32_t* bound = sh.bound + a.group_offset;
  const int32_t zero_lo = bound[0], zero_hi = bound[a.g_local];
  const bool whole = a.shares == 0;
  if (!whole && blockIdx.x == 0 && a.d_bias != nullptr) {
    // what the second kernel needs to know
    int32_t* head = reinterpret_cast<int32_t*>(a.parts);
    if (threadIdx.x == 0) head[0] = rows;
    for (int j = threadIdx.x; j <= a.g_local; j += kActThreads) head[1 + j] = bound[j];
  }
  const int64_t units = static_cast<int64_t>(whole ? a.g_local + 2 : a.shares) * col_blocks;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int32_t share = static_cast<int32_t>(u / col_blocks);
    const int64_t col0 = (u - static_cast<int64_t>(share) * col_blocks) * (W * 8);
    int32_t r, end;
    int j = 0;
    if (whole) {
      // share: a local group, or the rows before or after them
      j = share < a.g_local ? share : 0;
      r = share < a.g_local ? bound[j] : (share == a.g_local ? 0 : zero_hi);
      end = share < a.g_local ? bound[j + 1] : (share == a.g_local ? zero_lo : L);
      if (share < a.g_local && r == end && a.d_bias != nullptr)
        for (int c = threadIdx.x; c < W * 8; c += kActThreads)
          if (col0 + c < n) a.d_bias[j * n + col0 + c] = 0.0f;
    } else {
      const int64_t from = static_cast<int64_t>(share) * rows;
      if (from >= L) continue;
      r = static_cast<int32_t>(from);
      end = L - r > rows ? r + rows : L;
      // the last group that starts at or before r: it has rows, where r is in a group
      for (int top = a.g_local; top - j > 1;) {
        const int mid = (j + top) >> 1;
        if (bound[mid] <= r) j = mid; else top = mid;
      }
    }
    while (r < end) {
      if (r < zero_lo || r >= zero_hi) {
        const int32_t hi = r < zero_lo && zero_lo < end ? zero_lo : end;
        const int64_t col = col0 + col_lane * 8;
        if (a.d_pre != nullptr && col < n)
          for (int64_t row = r + static_cast<int64_t>(row_lane); row < hi; row += kLanes)
            *reinterpret_cast<uint4*>(static_cast<bf16*>(a.d_pre) + row * n + col) = make_uint4(0, 0, 0, 0);
        r = hi;
        continue;
      }
      while (bound[j + 1] <= r) ++j;
      const int32_t hi = bound[j + 1] < end ? bound[j + 1] : end;
      float2 sum[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[e] = both(0.0f);
      act_bwd_rows<D, ACT, W>(a, r, hi, col0, ring, sum);
      r = hi;
      if (a.d_bias == nullptr) continue;
      __syncthreads();  // the sums of the rows before have been read
#pragma unroll
      for (int e = 0; e < 4; ++e)
        *reinterpret_cast<float2*>(&across[row_lane][col_lane * 8 + 2 * e]) = sum[e];
      __syncthreads();
      float* part = whole ? a.d_bias + j * n + col0
                          : a.parts + kPartsAt / 4 + (static_cast<int64_t>(share) + j) * n + col0;
      for (int c = threadIdx.x; c < W * 8; c += kActThreads) {
        if (col0 + c >= n) continue;
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < kLanes; ++i) s += across[i][c];
        part[c] = s;
      }
    }
  }
}

// A group's sums to its gradient: Q quads of columns a block, 256 / Q threads a quad that each take every so many shares in
// order.  Eight quads are for few groups and columns, where a sum would otherwise be one block's long way
// (both kernels, us, 32 / 8 quads: 20000 x 128 13.2 / 9.2, 509 x 4096 7.9 / 7.4, but 4096 x 4096 in 16 groups 23.2 / 24.9).
template <int Q>
__global__ void __launch_bounds__(256) linear_bias_parts_kernel(const ActBwdArgs a) {
  constexpr int kCols = 4 * Q, kLanes = 256 / Q;
  __shared__ float4 across[8][Q];
  pdl_trigger();
  pdl_wait();
  const int quad = threadIdx.x % Q, part_lane = threadIdx.x / Q, warp = threadIdx.x >> 5;
  const int64_t n = a.n, col_blocks = (n + kCols - 1) / kCols;
  const int32_t* head = reinterpret_cast<const int32_t*>(a.parts);
  const float* parts = a.parts + kPartsAt / 4;
  const int32_t rows = head[0];
  const int64_t units = col_blocks * a.g_local;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int64_t j = u / col_blocks, col = (u - j * col_blocks) * kCols + quad * 4;
    const int32_t lo = head[1 + j], hi = head[2 + j];
    const int32_t first = lo / rows, last = hi > lo ? (hi - 1) / rows : first - 1;
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (col < n) {
#pragma unroll 8
      for (int32_t p = first + part_lane; p <= last; p += kLanes) {
        const float4 t = *reinterpret_cast<const float4*>(parts + (p + j) * n + col);
        v[0] += t.x, v[1] += t.y, v[2] += t.z, v[3] += t.w;
      }
    }
#pragma unroll
    for (int d = Q; d < 32; d <<= 1)
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], d);
    __syncthreads();
    if ((threadIdx.x & 31) < Q) across[warp][quad] = make_float4(v[0], v[1], v[2], v[3]);
    __syncthreads();
    if (threadIdx.x < Q && col < n) {
      float2 s[2];
      widen(across[0][quad], s);
#pragma unroll
      for (int i = 1; i < 8; ++i) {
        const float4 t = across[i][quad];
        s[0] = add2(s[0], make_float2(t.x, t.y));
        s[1] = add2(s[1], make_float2(t.z, t.w));
      }
      store4(a.d_bias + j * n + col, s);
    }
  }
}

constexpr int kFewUnits = 64;  // of 128 columns and a group

// Whether a block takes a whole group: groups enough for all SMs, at most 2048 rows of all of them, or few rows (us whole / shares, gelu: 8 x 136
// 2.5 / 4.0, 200 x 4096 5.0 / 5.5, 32 x 136 in 64 groups 2.9 / 12, 509 x 1024 in 16 4.6 / 6.2, 1024 x 1024 in 4 6.1 / 6.8, but 509 x 1024 6.5 /
// 4.8, 2000 x 4096 in 4 16 / 14).  The host does not know the groups' rows: these are even groups.  With all rows in one of them, its blocks have
// all of the work (us even / all in one / as one weight, by shares; inputs in L2: 2048 x 1024 in 64 5.5 / 50 / 6.8, 2048 x 4096 in 16 12 / 66 / 12,
// 1000 x 1024 in 4 5.2 / 11 / 5.7, 1024 x 14336 in 8 20 / 21 / 18): 2048 rows are the bound of that.
bool whole_groups(int64_t m, int64_t n, int32_t g_local) {
  return m <= 2048 && ((n + 63) / 64 * g_local >= 304 || m <= 256 * static_cast<int64_t>(g_local < 4 ? g_local : 4));
}

template <class D, int ACT, int W>
cudaError_t go(ActBwdArgs a, cudaStream_t stream) {
  constexpr size_t smem = static_cast<size_t>(kActStages) * kActThreads *
                          (RowPiece<D, W>::kBytes + (ACT != RD_ACT_NONE ? RowPiece<bf16, W>::kBytes : 0));
  static std::atomic<bool> set[64];
  int dev = 0;
  const cudaError_t e = allow_smem(linear_act_bwd_kernel<D, ACT, W>, smem, set, &dev);
  if (e != cudaSuccess) return e;
  const int32_t col_blocks = ceil_div(a.n, W * 8);
  // a whole group a turn, on as many blocks as run at once (each finds the boundaries once), or a share a block
  int64_t blocks = static_cast<int64_t>(a.g_local + 2) * col_blocks;
  if (blocks > kActSlots<ACT>) blocks = kActSlots<ACT>;
  a.shares = 0;
  if (!whole_groups(a.m, a.n, a.g_local)) {
    a.shares = kActSlots<ACT> / col_blocks;
    const int32_t most = ceil_div(a.m, kActLeastRows);
    if (a.shares > most) a.shares = most;
    if (a.shares < 1) a.shares = 1;
    blocks = static_cast<int64_t>(a.shares) * col_blocks;
  }
  return launch_pdl(linear_act_bwd_kernel<D, ACT, W>, dim3(static_cast<unsigned>(blocks)), kActThreads, smem, 1, stream, a);
}

template <class D, int ACT>
cudaError_t by_width(const ActBwdArgs& a, int sms, cudaStream_t stream) {
  cudaError_t e;
  const bool whole = whole_groups(a.m, a.n, a.g_local);
  // Whole groups: 128 columns a block, whose units are two turns of the blocks (2048 x 1024, 64 groups: 8.0 us; 64 columns and four turns
  // 9.7).  256 where units are many and groups short (us 128 / 256: 64 x 4096 in 64 groups 8.2 / 5.6, 256 x 14336 in 64 35 / 20, 1000 x
  // 2048 in 64 9.7 / 8.3, but 2048 x 2048 in 16 12 / 17).  32 or, of many, 64 columns where a group's rows are more than a few turns (us 32 / 64 /
  // 128: 200 x 4096 5.0 / 5.8 / 8, 509 x 136 in 4 4.0 / 4.9, 100 x 14336 7.0 / 5.5 / 6.5).
  const bool wide = a.m <= 32 * static_cast<int64_t>(a.g_local) && static_cast<int64_t>(a.n) * a.g_local >= 128 * 608;
  const bool tall = whole && a.m <= 1024 && a.m > 64 * static_cast<int64_t>(a.g_local);
  if (tall && a.n <= 4096) e = go<D, ACT, 4>(a, stream);
  else if (tall || a.n <= 64) e = go<D, ACT, 8>(a, stream);
  else if ((whole && !wide) || a.n <= 128) e = go<D, ACT, 16>(a, stream);
  else e = go<D, ACT, 32>(a, stream);
  if (e != cudaSuccess || whole || a.d_bias == nullptr) return e;
  const int64_t quads = a.n / 4, most = static_cast<int64_t>(sms) * 8;
  const bool few = (quads + 31) / 32 * a.g_local <= kFewUnits;
  const int64_t units = (few ? (quads + 7) / 8 : (quads + 31) / 32) * a.g_local;
  const dim3 grid(static_cast<unsigned>(units < most ? units : most));
  return few ? launch_pdl(linear_bias_parts_kernel<8>, grid, 256, 0, 1, stream, a)
             : launch_pdl(linear_bias_parts_kernel<32>, grid, 256, 0, 1, stream, a);
}

}  // namespace

// room for the sums of every share and group (no more shares than go() makes: its widths, and the most slots)
int64_t linear_act_bwd_bytes(int64_t m, int64_t n, int32_t g_local) {
  if (whole_groups(m, n, g_local)) return 0;
  const int64_t width = n <= 64 ? 64 : (n <= 128 ? 128 : 256);
  int64_t shares = kActMostSlots / ((n + width - 1) / width > 0 ? (n + width - 1) / width : 1);
  const int64_t most = (m + kActLeastRows - 1) / kActLeastRows;
  if (shares > most) shares = most;
  if (shares < 1) shares = 1;
  return kPartsAt + 4 * n * (shares + g_local);
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
