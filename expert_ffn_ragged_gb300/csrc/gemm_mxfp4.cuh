// gemm_mxfp4.cuh -- the persistent grouped product over 4-bit microscaled operands.
//
//   out[i, :] = sum_k a[i, k] * b[j, :, k]   for rows i of local group j, both operands E2M1 codes
//   with one E8M0 scale per 32 elements of k, f32 accumulation (tcgen05.mma kind::mxf4).
//
// The schedule (group boundaries, bands of m-tiles, the last m-tile of a group shifted back to its
// end) is that of the bf16 products (gemm_kernel.cuh); what differs:
//   * 128 bytes of a row are 256 elements of k, which the MMA takes in four steps of 64.  Both
//     operands are K-major.  A ring stage of the pair variant holds two such blocks: the MMA thread
//     then waits and commits once per 8 MMAs (768 cycles of tensor work).  With a wait for the
//     operands, one for the scales and two commits per 4 MMAs it was the thread's own instructions
//     that bound the kernel (855 cycles per 256 elements of k instead of 384, whatever else was
//     left out).  For the same reason the scales' arrival counts on the operands' barrier;
//   * a tile is 192 columns wide (96 gate + 96 up columns with the GLU).  Tensor memory has 512
//     columns: two 192-column accumulators leave 128 for the scales, two 256-column ones would
//     leave none;
//   * the scales keep their natural row-major layout in global memory: TMA brings 32 bytes a row
//     (1024 elements of k) of the tile's 128 + 192 rows into shared memory, and four warps, one
//     per lane quarter, move them from there to tensor memory, transposed on the way: the tensor
//     core wants, for 128 elements of k, row r's four scale bytes in lane r % 32 of column r / 32,
//     repeated in every lane quarter.  Every ring stage has scale columns of its own, so the scales
//     run as far ahead as the operands (with two slots of 512 elements for three such stages the
//     MMAs waited for them: 710 cycles per 256 elements).  No padding of groups and no packing of the
//     scales is needed, and the row shift of a group's last tile is free.  (Loaded straight from
//     global memory into registers and passed on through shared memory, the scales held the MMAs to
//     1350 cycles per 256 elements of k.)
// Warps: 0 operand producer, 1 MMA issuer, 2-9 epilogue, 10-13 scales, 14 scale producer.  Zero rows
// are written by the epilogue warps when their tiles are done.
//
// Bound and measured: large groups by the tensor cores (one pair MMA of 256 x 192 x 64 takes 96 cycles:
// 10.3 PFLOP/s at 2.07 GHz; the nominal dense rate, 13.5, is that of the 96-deep step, not used here)
// and, back to back, by the power limit: 32768 x 4096 x 14336 over 8 experts 605 us alone (6.4 PFLOP/s; with
// the GLU 566, with its 4-bit output 588), 640 to 680 in a loop at the power cap; of the 605, left out one
// after another, 100 go with the operands' copies, 65 with the output's stores, 400 are MMAs and tile
// padding.  Few rows an expert by the weights' bytes: 256 tokens top-8 of 128 experts, up 66 us (419 MB:
// 6.3 TB/s), down 39 us (214 MB: 5.5 TB/s; start and end of a launch, about 6 us, weigh more there).  One
// token: 12 us (64 tiles) and 8 us (176 tiles, two rounds of the 152 SMs), a chain of a few stages each.
#pragma once

#include "gemm_kernel.cuh"
#include "launch.h"
#include "moe_args.h"
#include "mxfp4.cuh"

namespace rd {

constexpr int k4BK = 256;       // elements of k in 128 bytes of a row
constexpr int k4BN = 192;       // output columns of a tile
constexpr int k4Half = k4BN / 2;
constexpr int k4Threads = 480;
constexpr int k4ScaleWarps = 4;
constexpr int k4RawK = 1024;    // elements of k of a shared-memory scale slot (32 scale bytes a row)
constexpr int k4RawSlots = 3;
// Tensor memory: two accumulators, then the scale columns of each stage: per word (128 elements of
// k) 4 columns for A's 128 rows, then per word 6 for B's 192.
constexpr int k4ScaleCol = 2 * k4BN;
constexpr int k4WordColsA = kBM / 32;
constexpr int k4WordColsB = k4BN / 32;

enum Gemm4Epi : int { k4EpiNone = 0, k4EpiGlu = 1, k4EpiGluQuant = 2 };

// Tiles: of 256 rows on a CTA pair, of 128 rows on one CTA, or of 32 rows on one CTA for groups of few
// rows.  The last is the 128-row MMA with rows of its own in the last lane quarter only: its A copies are
// a quarter as large, which makes room for six stages of B in place of four, and what the MMA reads as
// the other 96 rows is whatever lies before them in shared memory (any bits are E2M1 numbers, and no warp
// looks at those accumulator rows).  Against 128-row tiles, a layer's replays in a graph: one token 28.4 ->
// 26.1 us, 256 tokens 122.1 -> 120.7.
enum Gemm4Variant : int { k4Pair = 0, k4Single = 1, k4Few = 2 };

struct Gemm4Args {
  const int32_t* group_sizes;
  const int32_t* limit;
  int32_t* status;
  void* out;
  uint8_t* out_scales;
  int32_t m;
  int32_t kc;            // contraction length (elements)
  int32_t n_out;         // output columns (n, or n / 2 with the GLU)
  int32_t out_scale_width;
  int32_t g_total;
  int32_t group_offset;
  int32_t g_local;
  int32_t n_tiles;
  int32_t dw_m_tiles;    // unused (schedule)
  int32_t band_tiles;
  uint64_t timeout_ns;
};

// operands and their scales; boxes: a 128 rows, b 96 rows (of 128 bytes; scales: of 32)
struct Gemm4Maps {
  CUtensorMap a, b, a_scales, b_scales;
};

template <int VAR>
struct Tile4Cfg {
  static constexpr bool kPair = VAR == k4Pair;
  static constexpr bool kFew = VAR == k4Few;
  static constexpr int kStagesN = kPair ? 3 : (kFew ? 6 : 4);
  static constexpr int kSub = kPair ? 2 : 1;            // 256-element blocks of a stage
  static constexpr int kMmaM = kPair ? 2 * kBM : kBM;
  static constexpr int kARows = kFew ? 32 : kBM;        // A rows held by one CTA
  static constexpr int kTileM = kPair ? 2 * kBM : kARows;
  static constexpr int kBRows = kPair ? k4Half : k4BN;  // B rows held by one CTA
  static constexpr int kSubA = kARows * 128;            // 16 KB, or 4 KB
  static constexpr int kSubB = kBRows * 128;            // 12 KB (pair) or 24 KB
  static constexpr int kStageA = kSub * kSubA;
  static constexpr int kStageB = kSub * kSubB;
  static constexpr int kStageBytes = kStageA + kStageB;
  // A after B where the MMA's first rows lie before it, else before
  static constexpr int kOffA = kFew ? kStagesN * kStageB : 0;
  static constexpr int kOffB = kFew ? 0 : kStagesN * kStageA;
  static constexpr int kRowsBefore = kBM - kARows;      // MMA rows that are not the tile's
  static constexpr int kRawA = kARows * 32;             // scales of A's rows in a slot, then B's
  static constexpr int kRawBytes = kRawA + k4BN * 32;
  static constexpr int kWords = 2 * kSub;              // scale words of a row per stage
  static constexpr int kColsA = kWords * k4WordColsA;  // scale columns of a stage: A's, then B's
  static constexpr int kCols = kColsA + kWords * k4WordColsB;
  static_assert(k4ScaleCol + kStagesN * kCols <= kTmemCols, "tensor memory");
};

template <int VAR>
struct alignas(128) Gemm4Shared {
  static constexpr int S = Tile4Cfg<VAR>::kStagesN;
  uint8_t raw[k4RawSlots][Tile4Cfg<VAR>::kRawBytes];  // first: TMA destinations (128-byte aligned)
  uint64_t full[S];
  uint64_t empty[S];
  uint64_t rfull[k4RawSlots];
  uint64_t rempty[k4RawSlots];
  uint64_t tfull[2];
  uint64_t tempty[2];
  uint64_t drain;
  uint32_t tmem_base;
  int32_t abort_flag;
  int32_t L;
  int32_t total_tiles;
  int32_t zero_lo;
  int32_t zero_hi;
  int32_t bound[kMaxGroups + 1];
  int32_t tile_start[kMaxGroups + 1];
  uint4 epi[kEpiWarps][32 * 4];
};

template <int VAR>
constexpr size_t gemm4_smem_bytes() {
  return 1024 + static_cast<size_t>(Tile4Cfg<VAR>::kStagesN) * Tile4Cfg<VAR>::kStageBytes +
         sizeof(Gemm4Shared<VAR>);
}

// Tile t, as decode_tile_view has it.  A role's tiles only ever move forward, so the group is searched
// from that of its last tile on (`hint`); the divisions are left out where a group is one m-tile
// high, as in decoding, or one band.
template <int VAR>
__device__ __forceinline__ Tile decode_tile4(const Gemm4Shared<VAR>& sh, const Gemm4Args& a, int t,
                                             int& hint) {
  constexpr int TM = Tile4Cfg<VAR>::kTileM;
  constexpr int kStageK = Tile4Cfg<VAR>::kSub * k4BK;
  int j = hint;
  if (sh.tile_start[j + 1] <= t) {
    int hi = a.g_local;  // tile_start[j] <= t < tile_start[hi]
    while (hi - j > 1) {
      const int mid = (j + hi) >> 1;
      if (sh.tile_start[mid] <= t) j = mid;
      else hi = mid;
    }
    hint = j;
  }
  Tile tl;
  tl.j = j;
  tl.rs = sh.bound[a.group_offset + j];
  tl.re = sh.bound[a.group_offset + j + 1];
  int u = t - sh.tile_start[j];
  const int mt = ceil_div(tl.re - tl.rs, TM);
  if (mt == 1) {
    tl.m_idx = 0;
    tl.n_idx = u;
  } else {
    int first = 0, bw = mt;
    if (mt > a.band_tiles) {
      const int per_band = a.band_tiles * a.n_tiles;
      const int band = u / per_band;
      u -= band * per_band;
      first = band * a.band_tiles;
      bw = min(a.band_tiles, mt - first);
    }
    tl.n_idx = u / bw;
    tl.m_idx = first + u - tl.n_idx * bw;
  }
  tl.row_load = tl.m_idx == mt - 1 ? tl.re - TM : tl.rs + tl.m_idx * TM;
  tl.nkb = (a.kc + kStageK - 1) / kStageK;  // stages of the tile
  return tl;
}

// First row of b[j] behind tile column c (0 .. 191): with the GLU the first half of the tile are
// gate rows, the second half the up rows of the same output columns.
template <bool GLU>
__device__ __forceinline__ int b_row_of(int n_idx, int c, int n_out) {
  if (!GLU) return n_idx * k4BN + c;
  return c < k4Half ? n_idx * k4Half + c : n_out + n_idx * k4Half + (c - k4Half);
}

// One lane waits for the warp (polls by all lanes end at different times and then wait for each other).
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                          uint64_t limit_ns, int lane) {
  int ok = 1;
  if (lane == 0) ok = ptx::mbar_wait_bounded(bar, parity, abort_flag, limit_ns) ? 1 : 0;
  return __shfl_sync(0xFFFFFFFFu, ok, 0) != 0;
}

template <int EPI, int VAR>
__global__ void __launch_bounds__(k4Threads, 1)
    grouped_gemm_mxfp4_kernel(const __grid_constant__ Gemm4Maps maps, const Gemm4Args args) {
  constexpr bool GLU = EPI != k4EpiNone;
  using Cfg = Tile4Cfg<VAR>;
  constexpr bool PAIR = Cfg::kPair;
  constexpr int S = Cfg::kStagesN;
  constexpr int TM = Cfg::kTileM;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sA = smem + Cfg::kOffA;
  uint8_t* sB = smem + Cfg::kOffB;
  Gemm4Shared<VAR>& sh = *reinterpret_cast<Gemm4Shared<VAR>*>(smem + S * Cfg::kStageBytes);

  // the same in every lane of a warp, which the compiler cannot see of threadIdx.x >> 5
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0);
  const int lane = threadIdx.x & 31;
  volatile int* abort_flag = &sh.abort_flag;
  // rank in the cluster of two along x; the even CTA issues the MMAs
  const uint32_t rank = PAIR ? blockIdx.x & 1u : 0u;
  const bool leader = rank == 0;
  const int unit = PAIR ? static_cast<int>(blockIdx.x >> 1) : static_cast<int>(blockIdx.x);
  const int units = PAIR ? static_cast<int>(gridDim.x >> 1) : static_cast<int>(gridDim.x);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      // the producer's arrival (with the copies' bytes) and those of the scale warps
      ptx::mbar_init(ptx::smem_addr(&sh.full[s]), 1 + (PAIR ? 2 : 1) * k4ScaleWarps);
      ptx::mbar_init(ptx::smem_addr(&sh.empty[s]), 1);
    }
    for (int s = 0; s < k4RawSlots; ++s) {
      ptx::mbar_init(ptx::smem_addr(&sh.rfull[s]), 1);
      ptx::mbar_init(ptx::smem_addr(&sh.rempty[s]), k4ScaleWarps);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(ptx::smem_addr(&sh.tfull[b]), 1);
      ptx::mbar_init(ptx::smem_addr(&sh.tempty[b]), PAIR ? 2 * kEpiWarps : kEpiWarps);
    }
    ptx::mbar_init(ptx::smem_addr(&sh.drain), 1);
    sh.abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 0 && lane == 0 && args.kc > 0) {
    ptx::prefetch_tmap(&maps.a);
    ptx::prefetch_tmap(&maps.b);
    ptx::prefetch_tmap(&maps.a_scales);
    ptx::prefetch_tmap(&maps.b_scales);
  }
  if (warp == 1) {
    if (PAIR) {
      ptx::tmem_alloc_pair(ptx::smem_addr(&sh.tmem_base), kTmemCols);
      ptx::tmem_relinquish_pair();
    } else {
      ptx::tmem_alloc(ptx::smem_addr(&sh.tmem_base), kTmemCols);
      ptx::tmem_relinquish();
    }
  }
  // everything above touches no memory of the stream's earlier work
  pdl_trigger();
  pdl_wait();
  if (warp == 2) build_schedule<kOpFwd, TM>(sh, args, lane);
  ptx::tc_fence_before();
  __syncthreads();
  if (PAIR) ptx::cluster_sync();
  ptx::tc_fence_after();

  const int total = sh.total_tiles;
  const uint64_t tlimit = args.timeout_ns;
  int group = 0;  // of this role's last tile

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      uint32_t pend_mask = 0, pend_par = 0;
      bool ok = true;
      for (int t = unit; t < total && ok; t += units) {
        const Tile tl = decode_tile4<VAR>(sh, args, t, group);
        const int arow = tl.row_load + static_cast<int>(rank) * kBM;
        // the 96-row boxes of b: one per CTA of a pair, two on a single CTA
        const int brow0 = b_row_of<GLU>(tl.n_idx, 0, args.n_out);
        const int brow1 = b_row_of<GLU>(tl.n_idx, k4Half, args.n_out);
        for (int kb = 0; kb < tl.nkb; ++kb) {
          const int k0 = kb * Cfg::kSub * k4BK;
          const uint32_t fb_local = ptx::smem_addr(&sh.full[stage]);
          const uint32_t fb = PAIR ? ptx::map_to_rank(fb_local, 0) : fb_local;
          const uint32_t a_dst = ptx::smem_addr(sA + stage * Cfg::kStageA);
          const uint32_t b_dst = ptx::smem_addr(sB + stage * Cfg::kStageB);
          // the last stage of a row may hold fewer blocks
          const int left = (args.kc - k0 + k4BK - 1) / k4BK;
          const int subs = left < Cfg::kSub ? left : Cfg::kSub;
          if (!ptx::mbar_wait_bounded(ptx::smem_addr(&sh.empty[stage]), phase ^ 1, abort_flag, tlimit)) {
            ok = false;
            break;
          }
          pend_mask &= ~(1u << stage);
          if (rank == 0)
            ptx::mbar_arrive_expect_tx(fb_local, (PAIR ? 2 : 1) * subs * (Cfg::kSubA + Cfg::kSubB));
#pragma unroll
          for (int i = 0; i < Cfg::kSub; ++i) {
            if (i >= subs) break;
            const int x = k0 / 4 + i * 64;  // four codes a map element
            if (PAIR) {
              ptx::tma_load_2d_pair(a_dst + i * Cfg::kSubA, &maps.a, fb, x, arow);
              ptx::tma_load_3d_pair(b_dst + i * Cfg::kSubB, &maps.b, fb, x, rank == 0 ? brow0 : brow1, tl.j);
            } else {
              ptx::tma_load_2d(a_dst, &maps.a, fb, x, arow);
              ptx::tma_load_3d(b_dst, &maps.b, fb, x, brow0, tl.j);
              ptx::tma_load_3d(b_dst + k4Half * 128, &maps.b, fb, x, brow1, tl.j);
            }
          }
          pend_mask |= 1u << stage;
          pend_par = (pend_par & ~(1u << stage)) | (phase << stage);
          if (++stage == S) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      // Leave only once every fill has been consumed.  Unwinding, a fill's barrier may never
      // complete (it also counts the scale warps, and in a pair the even CTA's holds the odd CTA's
      // copies): the copies in flight get a grace period instead.
      if (!*abort_flag) {
        for (int s = 0; s < S; ++s)
          if (pend_mask & (1u << s))
            ptx::mbar_wait_bounded(ptx::smem_addr(&sh.empty[s]), (pend_par >> s) & 1u, abort_flag, kDrainNs);
      }
      if (*abort_flag) {
        const uint64_t t0 = ptx::global_timer_ns();
        while (ptx::global_timer_ns() - t0 < kGraceNs) __nanosleep(1000);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    // The whole warp walks the loop, so that what the MMAs take (descriptors, tensor-memory
    // addresses) is known to be the same in every lane and stays in uniform registers; one elected
    // lane issues.  A wait that gives up only raises the abort flag: the MMAs after it compute on
    // whatever is there, and the loop is left at the next tile.
    if (leader) {
      constexpr uint32_t idesc0 = ptx::idesc_mxfp4_f32(Cfg::kMmaM, k4BN, 0);
      constexpr uint32_t idesc2 = ptx::idesc_mxfp4_f32(Cfg::kMmaM, k4BN, 2);
      // operand descriptors of stage 0; a stage, and a K step of 32 bytes, move the address field
      const uint64_t a_desc0 = ptx::sw128_desc(ptx::smem_addr(sA) - Cfg::kRowsBefore * 128, 16, 1024);
      const uint64_t b_desc0 = ptx::sw128_desc(ptx::smem_addr(sB), 16, 1024);
      const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, sh.tmem_base, 0);
      const int tiles = __shfl_sync(0xFFFFFFFFu, total, 0);
      int stage = 0, acc = 0;
      uint32_t acc_phase = 0, full_phase = 0;
      // every tile has the same stages, so none need be decoded here
      const int nkb = (args.kc + Cfg::kSub * k4BK - 1) / (Cfg::kSub * k4BK);
      for (int t = unit; t < tiles && nkb > 0; t += units) {
        ptx::mbar_wait_bounded_cluster(ptx::smem_addr(&sh.tempty[acc]), acc_phase ^ 1, abort_flag, tlimit);
        __syncwarp();
        if (__any_sync(0xFFFFFFFFu, *abort_flag != 0)) break;
        const uint32_t d_tmem = tmem + static_cast<uint32_t>(acc * k4BN);
        for (int kb = 0; kb < nkb; ++kb) {
          const uint64_t ad = a_desc0 + static_cast<uint64_t>(stage * (Cfg::kStageA >> 4));
          const uint64_t bd = b_desc0 + static_cast<uint64_t>(stage * (Cfg::kStageB >> 4));
          const uint32_t sfa = tmem + k4ScaleCol + static_cast<uint32_t>(stage * Cfg::kCols);
          const uint32_t sfb = sfa + Cfg::kColsA;
          constexpr int kSteps = 4 * Cfg::kSub;
          const int left = (args.kc - kb * Cfg::kSub * k4BK + 63) / 64;
          const int steps = left < kSteps ? left : kSteps;
          ptx::mbar_wait_bounded_cluster(ptx::smem_addr(&sh.full[stage]), full_phase, abort_flag, tlimit);
          __syncwarp();
          ptx::tc_fence_after();
          if (ptx::elect_one()) {
            auto mma = [&](int kk, uint32_t accum) {
              const uint64_t ak = ad + (kk >> 2) * (Cfg::kSubA >> 4) + (kk & 3) * 2;
              const uint64_t bk = bd + (kk >> 2) * (Cfg::kSubB >> 4) + (kk & 3) * 2;
              const uint32_t fa = sfa + (kk >> 1) * k4WordColsA, fb = sfb + (kk >> 1) * k4WordColsB;
              const uint32_t id = (kk & 1) ? idesc2 : idesc0;
              if (PAIR) ptx::tc_mma_mxfp4_pair(d_tmem, ak, bk, id, fa, fb, accum);
              else ptx::tc_mma_mxfp4(d_tmem, ak, bk, id, fa, fb, accum);
            };
            if (steps == kSteps) {
              mma(0, kb > 0 ? 1u : 0u);
#pragma unroll
              for (int kk = 1; kk < kSteps; ++kk) mma(kk, 1u);
            } else {
#pragma unroll 1
              for (int kk = 0; kk < steps; ++kk) mma(kk, (kb > 0 || kk > 0) ? 1u : 0u);
            }
            if (PAIR) ptx::tc_commit_pair(ptx::smem_addr(&sh.empty[stage]), 0x3);
            else ptx::tc_commit(ptx::smem_addr(&sh.empty[stage]));
          }
          __syncwarp();
          if (++stage == S) {
            stage = 0;
            full_phase ^= 1;
          }
        }
        if (ptx::elect_one()) {
          if (PAIR) ptx::tc_commit_pair(ptx::smem_addr(&sh.tfull[acc]), 0x3);
          else ptx::tc_commit(ptx::smem_addr(&sh.tfull[acc]));
        }
        __syncwarp();
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1;
      }
      if (*abort_flag) {
        // every MMA issued has completed before TMEM is freed
        volatile int no_abort = 0;
        if (ptx::elect_one()) {
          if (PAIR) ptx::tc_commit_pair(ptx::smem_addr(&sh.drain), 0x1);
          else ptx::tc_commit(ptx::smem_addr(&sh.drain));
        }
        ptx::mbar_wait_bounded(ptx::smem_addr(&sh.drain), 0, &no_abort, kDrainNs);
      }
    }
    __syncwarp();
  } else if (warp < 2 + kEpiWarps) {
    // ------------------------------------------------------------ epilogue
    const int e = warp - 2;
    const int q = warp & 3;
    const int half = e >> 2;
    constexpr int tile_w = GLU ? k4Half : k4BN;
    constexpr int kChunks = tile_w / 32;
    uint4* stg = sh.epi[e];
    const uint32_t tempty_leader = PAIR ? ptx::map_to_rank(ptx::smem_addr(&sh.tempty[0]), 0) : 0u;
    const int sr = lane >> 2;
    const int piece = lane & 3;
    __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(args.out);
    uint8_t* out_q = reinterpret_cast<uint8_t*>(args.out);
    const int64_t q_row_bytes = args.n_out / 2;
    int acc = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    for (int t = unit; t < total; t += units) {
      const Tile tl = decode_tile4<VAR>(sh, args, t, group);
      const int wrow0 = tl.row_load + static_cast<int>(rank) * kBM + q * 32 - Cfg::kRowsBefore;
      const int lo = tile_store_lo(tl, TM), hi = tile_store_hi(tl);
      const int col0 = tl.n_idx * tile_w;
      // this lane's 32 columns of its row to global memory, through a transpose (8 rows x 64
      // contiguous bytes a store)
      auto emit = [&](const uint32_t (&p)[16], int col) {
#pragma unroll
        for (int v = 0; v < 4; ++v)
          stg[lane * 4 + (v ^ ((lane >> 1) & 3))] =
              make_uint4(p[4 * v], p[4 * v + 1], p[4 * v + 2], p[4 * v + 3]);
        __syncwarp();
#pragma unroll
        for (int it = 0; it < 4; ++it) {
          const int rl = it * 8 + sr;
          const uint4 val = stg[rl * 4 + (piece ^ ((rl >> 1) & 3))];
          const int row = wrow0 + rl;
          const int c = col + piece * 8;
          if (row >= lo && row < hi && c + 8 <= args.n_out)
            *reinterpret_cast<uint4*>(out + static_cast<int64_t>(row) * args.n_out + c) = val;
        }
        __syncwarp();
      };
      // the same columns as a 4-bit block: 16 bytes of codes and a scale byte
      auto emit_quant = [&](const float (&h)[32], int col) {
        uint32_t amax = 0;
#pragma unroll
        for (int i = 0; i < 32; ++i) amax = max(amax, __float_as_uint(h[i]) & 0x7FFFFFFFu);
        const uint32_t sb = mx_scale_byte(amax);
        const float inv = mx_inverse(sb);
        uint32_t codes[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float f[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] = h[8 * j + i] * inv;
          codes[j] = sb == 255u ? 0u : mx_pack8(f);
        }
        const int row = wrow0 + lane;
        if (row >= lo && row < hi && col < args.n_out) {
          *reinterpret_cast<uint4*>(out_q + row * q_row_bytes + col / 2) =
              make_uint4(codes[0], codes[1], codes[2], codes[3]);
          args.out_scales[static_cast<int64_t>(row) * args.out_scale_width + col / kMxBlock] =
              static_cast<uint8_t>(sb);
        }
      };
      if (tl.nkb == 0) {
        const uint32_t z[16] = {0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
        float zf[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) zf[i] = 0.0f;
        for (int c = half; c < kChunks; c += 2) {
          if (EPI == k4EpiGluQuant) emit_quant(zf, col0 + c * 32);
          else emit(z, col0 + c * 32);
        }
        continue;
      }
      ok = warp_wait(ptx::smem_addr(&sh.tfull[acc]), acc_phase, abort_flag, tlimit, lane);
      if (!ok) break;
      ptx::tc_fence_after();
      const uint32_t tbase =
          sh.tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(acc * k4BN);
      // a group of a few rows leaves most warps' rows without an owner
      const bool any_rows = wrow0 < hi && wrow0 + 32 > lo;
#pragma unroll 1
      for (int c = half; c < kChunks && any_rows; c += 2) {
        if (GLU) {
          uint32_t g[32], u[32];
          ptx::tmem_load_32cols(tbase + c * 32, g);
          ptx::tmem_load_32cols(tbase + k4Half + c * 32, u);
          float h[32];
#pragma unroll
          for (int i = 0; i < 32; ++i)
            h[i] = glu_fwd_fast(__uint_as_float(g[i]), __uint_as_float(u[i]));
          if (EPI == k4EpiGluQuant) {
            emit_quant(h, col0 + c * 32);
          } else {
            uint32_t p[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) p[i] = pack_bf16x2(h[2 * i], h[2 * i + 1]);
            emit(p, col0 + c * 32);
          }
        } else {
          // Chunk by chunk.  All three read at once and the accumulator given back before the stores
          // was slower where the outputs dominate (131072 x 768 x 4096: 297 -> 334 us), as were stores
          // of 32 bytes a lane without the transpose (32768 x 4096 x 14336: 620 -> 680); whole 128-byte
          // lines (604 -> 613) and bulk tensor stores (603 -> 599, one token 26.4 -> 27.0) were no better.
          uint32_t v[32], p[16];
          ptx::tmem_load_32cols(tbase + c * 32, v);
#pragma unroll
          for (int i = 0; i < 16; ++i)
            p[i] = pack_bf16x2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
          emit(p, col0 + c * 32);
        }
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (PAIR && rank != 0)
          ptx::mbar_arrive_cluster_tmem(tempty_leader + static_cast<uint32_t>(acc * sizeof(uint64_t)));
        else
          ptx::mbar_arrive(ptx::smem_addr(&sh.tempty[acc]));
      }
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1;
    }
    // zero rows [0, zero_lo) and [zero_hi, L): whole rows of 16-byte units, shared by all CTAs
    auto zero = [&](uint8_t* base, int64_t row_bytes) {
      const int64_t per_row = row_bytes / 16;
      const int64_t units16 = (sh.zero_lo + static_cast<int64_t>(sh.L) - sh.zero_hi) * per_row;
      const int64_t skip = static_cast<int64_t>(sh.zero_hi - sh.zero_lo) * per_row;
      const int64_t lo16 = sh.zero_lo * per_row;
      for (int64_t i = static_cast<int64_t>(blockIdx.x) * (kEpiWarps * 32) + e * 32 + lane; i < units16;
           i += static_cast<int64_t>(gridDim.x) * (kEpiWarps * 32))
        reinterpret_cast<uint4*>(base)[i < lo16 ? i : i + skip] = make_uint4(0, 0, 0, 0);
    };
    if (EPI == k4EpiGluQuant) {
      zero(out_q, q_row_bytes);
      zero(args.out_scales, args.out_scale_width);
    } else {
      zero(out_q, static_cast<int64_t>(args.n_out) * 2);
    }
  } else if (warp == k4Threads / 32 - 1) {
    // ------------------------------------------------------------ scale producer
    // The tiles' scales, 1024 elements of k at a time, as far ahead as the slots allow: A's rows of
    // this CTA and all B rows of the tile.  (Issued together with the operands they arrived after
    // them, small rows that they are, and still had to be moved.)
    if (lane == 0) {
      int slot = 0;
      uint32_t phase = 0, pend_mask = 0, pend_par = 0;
      bool ok = true;
      for (int t = unit; t < total && ok; t += units) {
        const Tile tl = decode_tile4<VAR>(sh, args, t, group);
        const int arow = tl.row_load + static_cast<int>(rank) * kBM;
        const int brow0 = b_row_of<GLU>(tl.n_idx, 0, args.n_out);
        const int brow1 = b_row_of<GLU>(tl.n_idx, k4Half, args.n_out);
        for (int k0 = 0; k0 < args.kc; k0 += k4RawK) {
          ok = ptx::mbar_wait_bounded(ptx::smem_addr(&sh.rempty[slot]), phase ^ 1, abort_flag, tlimit);
          if (!ok) break;
          const uint32_t rb = ptx::smem_addr(&sh.rfull[slot]);
          const uint32_t dst = ptx::smem_addr(sh.raw[slot]);
          ptx::mbar_arrive_expect_tx(rb, Cfg::kRawBytes);
          const int x = k0 / (2 * kMxBlock);  // two scale bytes a map element
          ptx::tma_load_2d(dst, &maps.a_scales, rb, x, arow);
          ptx::tma_load_3d(dst + Cfg::kRawA, &maps.b_scales, rb, x, brow0, tl.j);
          ptx::tma_load_3d(dst + Cfg::kRawA + k4Half * 32, &maps.b_scales, rb, x, brow1, tl.j);
          pend_mask |= 1u << slot;
          pend_par = (pend_par & ~(1u << slot)) | (phase << slot);
          if (++slot == k4RawSlots) {
            slot = 0;
            phase ^= 1;
          }
        }
      }
      // leave only once the last copy of each slot has landed
      volatile int no_abort = 0;
      for (int s = 0; s < k4RawSlots; ++s)
        if (pend_mask & (1u << s))
          ptx::mbar_wait_bounded(ptx::smem_addr(&sh.rfull[s]), (pend_par >> s) & 1u, &no_abort, kDrainNs);
    }
  } else {
    // ------------------------------------------------------------ scales
    // Each of the four warps writes one lane quarter of tensor memory, which repeats the scales of
    // all rows: lane l holds those of rows l, 32 + l, ...  A raw row is 32 bytes, two halves of 16
    // that the copy's 32-byte swizzle exchanges in every second group of four rows, which makes
    // the reads below free of bank conflicts.
    const uint32_t full0 = PAIR ? ptx::map_to_rank(ptx::smem_addr(&sh.full[0]), 0)
                                : ptx::smem_addr(&sh.full[0]);
    const uint32_t col0 = sh.tmem_base + (static_cast<uint32_t>((warp & 3) * 32) << 16) + k4ScaleCol;
    constexpr int kW = Cfg::kWords;
    constexpr int kStageK = Cfg::kSub * k4BK;
    constexpr int kRowsL = (kBM + k4BN) / 32;  // rows of a lane
    int raw_slot = 0, stage = 0;
    uint32_t raw_phase = 0, phase = 0;
    bool ok = true;
    for (int t = unit; t < total && ok; t += units) {
      const Tile tl = decode_tile4<VAR>(sh, args, t, group);
      for (int kb = 0; kb < tl.nkb; ++kb) {
        const int k0 = kb * kStageK;
        if (k0 % k4RawK == 0) {
          ok = warp_wait(ptx::smem_addr(&sh.rfull[raw_slot]), raw_phase, abort_flag, tlimit, lane);
          if (!ok) break;
        }
        const int at = (k0 % k4RawK) / kMxBlock;  // first byte of the stage in a raw row
        const uint8_t* src = sh.raw[raw_slot] + lane * 32 + ((at ^ ((lane << 2) & 16)));
        uint32_t v[kRowsL][kW];
#pragma unroll
        for (int i = 0; i < kRowsL; ++i) {
          if (i < Cfg::kRowsBefore / 32) {
#pragma unroll
            for (int w = 0; w < kW; ++w) v[i][w] = 0;
          } else if constexpr (kW == 4) {
            const uint4 x = *reinterpret_cast<const uint4*>(src + i * 32 * 32);
            v[i][0] = x.x;
            v[i][1] = x.y;
            v[i][2] = x.z;
            v[i][3] = x.w;
          } else {
            const uint2 x = *reinterpret_cast<const uint2*>(src + (i - Cfg::kRowsBefore / 32) * 32 * 32);
            v[i][0] = x.x;
            v[i][1] = x.y;
          }
        }
        if ((k0 + kStageK) % k4RawK == 0 || kb == tl.nkb - 1) {
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(&sh.rempty[raw_slot]));
          if (++raw_slot == k4RawSlots) {
            raw_slot = 0;
            raw_phase ^= 1;
          }
        }
        // bytes past the end of k meet zero operands: they must not be NaN
        const int valid = (args.kc - k0) / kMxBlock;
        if (valid < 4 * kW) {
#pragma unroll
          for (int w = 0; w < kW; ++w) {
            const int nb = valid - 4 * w;
            const uint32_t keep = nb >= 4 ? 0xFFFFFFFFu : (nb <= 0 ? 0u : (1u << (8 * nb)) - 1u);
#pragma unroll
            for (int i = 0; i < kRowsL; ++i) v[i][w] &= keep;
          }
        }
        // the stage's columns, in the order of tensor memory
        uint32_t c[Cfg::kCols];
#pragma unroll
        for (int w = 0; w < kW; ++w) {
#pragma unroll
          for (int i = 0; i < k4WordColsA; ++i) c[w * k4WordColsA + i] = v[i][w];
#pragma unroll
          for (int i = 0; i < k4WordColsB; ++i)
            c[Cfg::kColsA + w * k4WordColsB + i] = v[k4WordColsA + i][w];
        }
        // free once the stage's previous MMAs are done, as for the producer
        ok = warp_wait(ptx::smem_addr(&sh.empty[stage]), phase ^ 1, abort_flag, tlimit, lane);
        if (!ok) break;
        ptx::tc_fence_after();
        const uint32_t col = col0 + static_cast<uint32_t>(stage * Cfg::kCols);
        if constexpr (kW == 4) {
          ptx::tmem_store_32cols(col, c);
          ptx::tmem_store_8cols(col + 32, c + 32);
        } else {
          ptx::tmem_store_16cols(col, c);
          ptx::tmem_store_4cols(col + 16, c + 16);
        }
        ptx::tmem_wait_stores();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          const uint32_t b = full0 + static_cast<uint32_t>(stage * sizeof(uint64_t));
          if (PAIR) ptx::mbar_arrive_cluster_tmem(b);
          else ptx::mbar_arrive(b);
        }
        if (++stage == S) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (PAIR) ptx::cluster_sync();
  if (warp == 1) {
    ptx::tc_fence_after();
    if (PAIR) ptx::tmem_dealloc_pair(sh.tmem_base, kTmemCols);
    else ptx::tmem_dealloc(sh.tmem_base, kTmemCols);
  }
  if (threadIdx.x == 0 && sh.abort_flag && args.status != nullptr)
    atomicOr(args.status, RD_STATUS_TIMEOUT);
}

}  // namespace rd
