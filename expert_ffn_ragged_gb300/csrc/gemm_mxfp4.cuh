// gemm_mxfp4.cuh -- the persistent grouped product over 4-bit microscaled operands.
//
//   out[i, :] = sum_k a[i, k] * b[j, :, k]   for rows i of local group j, both operands E2M1 codes
//   with one E8M0 scale per 32 elements of k, f32 accumulation (tcgen05.mma kind::mxf4).
//
// The schedule (group boundaries, bands of m-tiles, the last m-tile of a group shifted back to its
// end) is that of the bf16 products (gemm_kernel.cuh); what differs:
//   * 128 bytes of a row are 256 elements of k, so one ring stage is 256 deep and the MMA takes it
//     in four steps of 64.  Both operands are K-major;
//   * a tile is 192 columns wide (96 gate + 96 up columns with the GLU).  Tensor memory has 512
//     columns: two 192-column accumulators leave 64 columns beside each for the scales, two
//     256-column ones would leave none;
//   * the scales of a tile are loaded in their natural row-major layout by two warps (16 bytes a
//     row: 512 elements of k), laid out in shared memory the way the tensor core reads them (per
//     128 rows and 128 elements of k: 32 rows of 16 bytes, row r's word at (r % 32) * 16 +
//     (r / 32) * 4), and copied to tensor memory by the MMA thread just ahead of the MMAs that use
//     them.  No padding of groups and no packing of the scales is needed, and the row shift of a
//     group's last tile is free.
// Warps: 0 TMA producer, 1 MMA issuer, 2-9 epilogue, 10-11 scales.  Zero rows are written by the
// epilogue warps when their tiles are done.
#pragma once

#include "gemm_kernel.cuh"
#include "moe_args.h"
#include "mxfp4.cuh"

namespace rd {

constexpr int k4BK = 256;       // elements of k per stage (128 bytes a row)
constexpr int k4BN = 192;       // output columns of a tile
constexpr int k4Half = k4BN / 2;
constexpr int k4Chunk = 512;    // elements of k per scale chunk (16 scale bytes a row)
constexpr int k4ScaleSlots = 4;  // scale chunks in shared memory
constexpr int k4ScaleWarps = 2;

enum Gemm4Epi : int { k4EpiNone = 0, k4EpiGlu = 1, k4EpiGluQuant = 2 };

struct Gemm4Args {
  const int32_t* group_sizes;
  const int32_t* limit;
  int32_t* status;
  const uint8_t* a_scales;  // [m, scale_width]
  const uint8_t* b_scales;  // [g_local, n, scale_width]
  void* out;
  uint8_t* out_scales;
  int32_t m;
  int32_t kc;            // contraction length (elements)
  int32_t n;             // rows of each b block
  int32_t n_out;         // output columns (n, or n / 2 with the GLU)
  int32_t scale_width;   // bytes of a scale row of a and b
  int32_t out_scale_width;
  int32_t g_total;
  int32_t group_offset;
  int32_t g_local;
  int32_t n_tiles;
  int32_t dw_m_tiles;    // unused (schedule)
  int32_t band_tiles;
  uint64_t timeout_ns;
};

template <bool PAIR>
struct Tile4Cfg {
  static constexpr int kStagesN = PAIR ? 6 : 4;
  static constexpr int kTileM = PAIR ? 2 * kBM : kBM;
  static constexpr int kBRows = PAIR ? k4Half : k4BN;  // B rows held by one CTA
  static constexpr int kStageA = kBM * 128;            // 16 KB
  static constexpr int kStageB = kBRows * 128;         // 12 KB (pair) or 24 KB
  static constexpr int kStageBytes = kStageA + kStageB;
};

constexpr int k4WordA = 512;             // A scales of 128 rows x 128 k
constexpr int k4WordB = 1024;            // B scales of 192 (256) rows x 128 k
constexpr int k4SlotBytes = 4 * (k4WordA + k4WordB);

template <bool PAIR>
struct alignas(128) Gemm4Shared {
  static constexpr int S = Tile4Cfg<PAIR>::kStagesN;
  uint8_t scales[k4ScaleSlots][k4SlotBytes];
  uint64_t full[S];
  uint64_t empty[S];
  uint64_t sfull[k4ScaleSlots];
  uint64_t sempty[k4ScaleSlots];
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

template <bool PAIR>
constexpr size_t gemm4_smem_bytes() {
  return 1024 + static_cast<size_t>(Tile4Cfg<PAIR>::kStagesN) * Tile4Cfg<PAIR>::kStageBytes +
         sizeof(Gemm4Shared<PAIR>);
}

template <bool PAIR>
__device__ __forceinline__ Tile decode_tile4(const Gemm4Shared<PAIR>& sh, const Gemm4Args& a, int t) {
  SchedView v;
  v.bound = sh.bound;
  v.tile_start = sh.tile_start;
  v.group_offset = a.group_offset;
  v.g_local = a.g_local;
  v.n_tiles = a.n_tiles;
  v.band_tiles = a.band_tiles;
  v.dw_m_tiles = 0;
  v.kc = a.kc;
  Tile tl = decode_tile_view<kOpFwd, Tile4Cfg<PAIR>::kTileM>(v, t);
  tl.nkb = (a.kc + k4BK - 1) / k4BK;
  return tl;
}

// First row of b[j] behind tile column c (0 .. 191): with the GLU the first half of the tile are
// gate rows, the second half the up rows of the same output columns.
template <bool GLU>
__device__ __forceinline__ int b_row_of(int n_idx, int c, int n_out) {
  if (!GLU) return n_idx * k4BN + c;
  return c < k4Half ? n_idx * k4Half + c : n_out + n_idx * k4Half + (c - k4Half);
}

template <int EPI, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1)
    grouped_gemm_mxfp4_kernel(const __grid_constant__ CUtensorMap tmap_a,
                              const __grid_constant__ CUtensorMap tmap_b, const Gemm4Args args) {
  constexpr bool GLU = EPI != k4EpiNone;
  using Cfg = Tile4Cfg<PAIR>;
  constexpr int S = Cfg::kStagesN;
  constexpr int TM = Cfg::kTileM;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sA = smem;
  uint8_t* sB = smem + S * Cfg::kStageA;
  Gemm4Shared<PAIR>& sh = *reinterpret_cast<Gemm4Shared<PAIR>*>(smem + S * Cfg::kStageBytes);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  volatile int* abort_flag = &sh.abort_flag;
  const uint32_t rank = PAIR ? ptx::cluster_ctarank() : 0u;
  const int unit = PAIR ? static_cast<int>(blockIdx.x >> 1) : static_cast<int>(blockIdx.x);
  const int units = PAIR ? static_cast<int>(gridDim.x >> 1) : static_cast<int>(gridDim.x);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      ptx::mbar_init(ptx::smem_addr(&sh.full[s]), 1);
      ptx::mbar_init(ptx::smem_addr(&sh.empty[s]), 1);
    }
    for (int s = 0; s < k4ScaleSlots; ++s) {
      ptx::mbar_init(ptx::smem_addr(&sh.sfull[s]), PAIR ? 2 * k4ScaleWarps : k4ScaleWarps);
      ptx::mbar_init(ptx::smem_addr(&sh.sempty[s]), 1);
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
    ptx::prefetch_tmap(&tmap_a);
    ptx::prefetch_tmap(&tmap_b);
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
  if (warp == 2) build_schedule<kOpFwd, TM>(sh, args, lane);
  ptx::tc_fence_before();
  __syncthreads();
  if (PAIR) ptx::cluster_sync();
  ptx::tc_fence_after();

  const int total = sh.total_tiles;
  const uint64_t tlimit = args.timeout_ns;

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      uint32_t pend_mask = 0, pend_par = 0;
      bool ok = true;
      for (int t = unit; t < total && ok; t += units) {
        const Tile tl = decode_tile4<PAIR>(sh, args, t);
        const int arow = tl.row_load + static_cast<int>(rank) * kBM;
        // the 96-row boxes of b: one per CTA of a pair, two on a single CTA
        const int brow0 = b_row_of<GLU>(tl.n_idx, PAIR ? static_cast<int>(rank) * k4Half : 0, args.n_out);
        const int brow1 = b_row_of<GLU>(tl.n_idx, k4Half, args.n_out);
        for (int kb = 0; kb < tl.nkb; ++kb) {
          const uint32_t fb_local = ptx::smem_addr(&sh.full[stage]);
          const uint32_t fb = PAIR ? ptx::map_to_rank(fb_local, 0) : fb_local;
          const uint32_t a_dst = ptx::smem_addr(sA + stage * Cfg::kStageA);
          const uint32_t b_dst = ptx::smem_addr(sB + stage * Cfg::kStageB);
          if (!ptx::mbar_wait_bounded(ptx::smem_addr(&sh.empty[stage]), phase ^ 1, abort_flag, tlimit)) {
            ok = false;
            break;
          }
          pend_mask &= ~(1u << stage);
          if (rank == 0) ptx::mbar_arrive_expect_tx(fb_local, (PAIR ? 2 : 1) * Cfg::kStageBytes);
          // 128 bytes of a row are 64 two-byte elements of the maps
          const int x = kb * 64;
          if (PAIR) {
            ptx::tma_load_2d_pair(a_dst, &tmap_a, fb, x, arow);
            ptx::tma_load_3d_pair(b_dst, &tmap_b, fb, x, brow0, tl.j);
          } else {
            ptx::tma_load_2d(a_dst, &tmap_a, fb, x, arow);
            ptx::tma_load_3d(b_dst, &tmap_b, fb, x, brow0, tl.j);
            ptx::tma_load_3d(b_dst + k4Half * 128, &tmap_b, fb, x, brow1, tl.j);
          }
          pend_mask |= 1u << stage;
          pend_par = (pend_par & ~(1u << stage)) | (phase << stage);
          if (++stage == S) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      // leave only once every fill has been consumed (or, unwinding, has landed; the odd CTA
      // of a pair cannot see its copies, which count on the even CTA's barrier: a grace period)
      volatile int no_abort = 0;
      for (int s = 0; s < S; ++s) {
        if (!(pend_mask & (1u << s))) continue;
        const uint32_t par = (pend_par >> s) & 1u;
        if (*abort_flag) {
          if (!PAIR || rank == 0)
            ptx::mbar_wait_bounded(ptx::smem_addr(&sh.full[s]), par, &no_abort, kDrainNs);
        } else {
          ptx::mbar_wait_bounded(ptx::smem_addr(&sh.empty[s]), par, &no_abort, kDrainNs);
        }
      }
      if (PAIR && rank != 0 && *abort_flag && pend_mask != 0) {
        const uint64_t t0 = ptx::global_timer_ns();
        while (ptx::global_timer_ns() - t0 < kGraceNs) __nanosleep(1000);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (rank == 0 && lane == 0) {
      constexpr uint32_t idesc0 = ptx::idesc_mxfp4_f32(TM, k4BN, 0);
      constexpr uint32_t idesc2 = ptx::idesc_mxfp4_f32(TM, k4BN, 2);
      int stage = 0, acc = 0, slot = 0;
      uint32_t acc_phase = 0, full_phase = 0, slot_phase = 0;
      uint32_t sbuf = 0;  // which 64-column gap the next block's scales go to
      bool ok = true;
      for (int t = unit; t < total && ok; t += units) {
        const Tile tl = decode_tile4<PAIR>(sh, args, t);
        if (tl.nkb == 0) continue;
        ok = ptx::mbar_wait_bounded_cluster(ptx::smem_addr(&sh.tempty[acc]), acc_phase ^ 1, abort_flag, tlimit);
        if (!ok) break;
        ptx::tc_fence_after();
        const uint32_t d_tmem = sh.tmem_base + static_cast<uint32_t>(acc * kBN);
        for (int kb = 0; kb < tl.nkb; ++kb) {
          const uint32_t a_addr = ptx::smem_addr(sA + stage * Cfg::kStageA);
          const uint32_t b_addr = ptx::smem_addr(sB + stage * Cfg::kStageB);
          const uint32_t s_addr = ptx::smem_addr(sh.scales[slot]) + (kb & 1) * 2 * (k4WordA + k4WordB);
          const uint32_t s_tmem = sh.tmem_base + k4BN + sbuf * kBN;
          const int left = args.kc - kb * k4BK;
          const int steps = left >= k4BK ? 4 : (left + 63) / 64;
          if ((kb & 1) == 0) {
            ok = PAIR ? ptx::mbar_wait_bounded_cluster(ptx::smem_addr(&sh.sfull[slot]), slot_phase, abort_flag, tlimit)
                      : ptx::mbar_wait_bounded(ptx::smem_addr(&sh.sfull[slot]), slot_phase, abort_flag, tlimit);
            if (!ok) break;
          }
          ok = ptx::mbar_wait_bounded(ptx::smem_addr(&sh.full[stage]), full_phase, abort_flag, tlimit);
          if (!ok) break;
          ptx::tc_fence_after();
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const uint32_t sw = s_addr + w * (k4WordA + k4WordB);
            auto cp = [&](uint32_t col, uint32_t saddr) {
              if (PAIR) ptx::tc_copy_scales_pair(s_tmem + col, ptx::scales_desc(saddr));
              else ptx::tc_copy_scales(s_tmem + col, ptx::scales_desc(saddr));
            };
            cp(w * 4, sw);
            cp(8 + w * 8, sw + k4WordA);
            cp(8 + w * 8 + 4, sw + k4WordA + 512);
          }
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            if (kk >= steps) break;
            const uint64_t ad = ptx::sw128_desc(a_addr + kk * 32, 16, 1024);
            const uint64_t bd = ptx::sw128_desc(b_addr + kk * 32, 16, 1024);
            const uint32_t sfa = s_tmem + (kk >> 1) * 4, sfb = s_tmem + 8 + (kk >> 1) * 8;
            const uint32_t accum = (kb > 0 || kk > 0) ? 1u : 0u;
            if (PAIR) ptx::tc_mma_mxfp4_pair(d_tmem, ad, bd, (kk & 1) ? idesc2 : idesc0, sfa, sfb, accum);
            else ptx::tc_mma_mxfp4(d_tmem, ad, bd, (kk & 1) ? idesc2 : idesc0, sfa, sfb, accum);
          }
          sbuf ^= 1;
          const bool chunk_end = (kb & 1) || kb == tl.nkb - 1;
          if (PAIR) {
            if (chunk_end) ptx::tc_commit_pair(ptx::smem_addr(&sh.sempty[slot]), 0x3);
            ptx::tc_commit_pair(ptx::smem_addr(&sh.empty[stage]), 0x3);
          } else {
            if (chunk_end) ptx::tc_commit(ptx::smem_addr(&sh.sempty[slot]));
            ptx::tc_commit(ptx::smem_addr(&sh.empty[stage]));
          }
          if (chunk_end && ++slot == k4ScaleSlots) {
            slot = 0;
            slot_phase ^= 1;
          }
          if (++stage == S) {
            stage = 0;
            full_phase ^= 1;
          }
        }
        if (!ok) break;
        if (PAIR) ptx::tc_commit_pair(ptx::smem_addr(&sh.tfull[acc]), 0x3);
        else ptx::tc_commit(ptx::smem_addr(&sh.tfull[acc]));
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1;
      }
      if (*abort_flag) {
        volatile int no_abort = 0;
        if (PAIR) ptx::tc_commit_pair(ptx::smem_addr(&sh.drain), 0x1);
        else ptx::tc_commit(ptx::smem_addr(&sh.drain));
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
      const Tile tl = decode_tile4<PAIR>(sh, args, t);
      const int wrow0 = tl.row_load + static_cast<int>(rank) * kBM + q * 32;
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
      ok = ptx::mbar_wait_bounded(ptx::smem_addr(&sh.tfull[acc]), acc_phase, abort_flag, tlimit);
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (!ok) break;
      ptx::tc_fence_after();
      const uint32_t tbase =
          sh.tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(acc * kBN);
#pragma unroll 1
      for (int c = half; c < kChunks; c += 2) {
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
          ptx::mbar_arrive_cluster(tempty_leader + static_cast<uint32_t>(acc * sizeof(uint64_t)));
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
  } else {
    // ------------------------------------------------------------ scales
    // Rows 0 .. 127 of the tile's 320 are A's (this CTA's half in a pair), the others B's.  A lane
    // holds five rows: 16 bytes of each are 512 elements of k.  The next chunk is loaded into
    // registers before the wait for its slot, so that global latency overlaps it.
    const int sw = warp - (2 + kEpiWarps);
    constexpr int kRows = 5;
    const uint32_t sfull0 = PAIR ? ptx::map_to_rank(ptx::smem_addr(&sh.sfull[0]), 0)
                                 : ptx::smem_addr(&sh.sfull[0]);
    int slot = 0;
    uint32_t phase = 0, pend_mask = 0, pend_par = 0;
    const int blocks = args.kc / kMxBlock;  // scale bytes of a row that count
    bool ok = true;
    for (int t = unit; t < total && ok; t += units) {
      const Tile tl = decode_tile4<PAIR>(sh, args, t);
      const uint8_t* src[kRows];
      uint32_t dst[kRows];
      uint32_t word[kRows];
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int r = sw * kRows * 32 + i * 32 + lane;
        if (r < kBM) {
          const int row = tl.row_load + static_cast<int>(rank) * kBM + r;
          src[i] = row >= 0 && row < args.m ? args.a_scales + static_cast<int64_t>(row) * args.scale_width : nullptr;
          dst[i] = (r & 31) * 16 + (r >> 5) * 4;
          word[i] = k4WordA;
        } else {
          const int c = r - kBM;
          const int row = b_row_of<GLU>(tl.n_idx, c, args.n_out);
          src[i] = row < args.n ? args.b_scales + (static_cast<int64_t>(tl.j) * args.n + row) * args.scale_width
                                : nullptr;
          dst[i] = (c >> 7) * 512 + (c & 31) * 16 + ((c >> 5) & 3) * 4;
          word[i] = k4WordB;
        }
      }
      const int chunks = (tl.nkb + 1) / 2;
      auto load = [&](int ch, uint4 (&v)[kRows]) {
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          v[i] = make_uint4(0, 0, 0, 0);
          if (src[i] != nullptr) v[i] = __ldg(reinterpret_cast<const uint4*>(src[i] + ch * 16));
        }
      };
      uint4 next[kRows];
      if (chunks > 0) load(0, next);
      for (int ch = 0; ch < chunks; ++ch) {
        uint4 v[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) v[i] = next[i];
        if (ch + 1 < chunks) load(ch + 1, next);
        // bytes past the end of k meet zero operands: they must not be NaN
        const int valid = blocks - ch * 16;
        if (valid < 16) {
          auto keep = [&](uint32_t x, int w) {
            const int nb = valid - 4 * w;
            return nb >= 4 ? x : (nb <= 0 ? 0u : x & ((1u << (8 * nb)) - 1u));
          };
#pragma unroll
          for (int i = 0; i < kRows; ++i)
            v[i] = make_uint4(keep(v[i].x, 0), keep(v[i].y, 1), keep(v[i].z, 2), keep(v[i].w, 3));
        }
        ok = ptx::mbar_wait_bounded(ptx::smem_addr(&sh.sempty[slot]), phase ^ 1, abort_flag, tlimit);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        pend_mask &= ~(1u << slot);
        uint8_t* base = sh.scales[slot];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          const uint32_t w4[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
          // a slot holds, per 128 elements of k, the words of A's rows, then those of B's
          uint8_t* p = base + (word[i] == k4WordA ? 0 : k4WordA) + dst[i];
#pragma unroll
          for (int w = 0; w < 4; ++w)
            *reinterpret_cast<uint32_t*>(p + w * (k4WordA + k4WordB)) = w4[w];
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          const uint32_t b = sfull0 + static_cast<uint32_t>(slot * sizeof(uint64_t));
          if (PAIR) ptx::mbar_arrive_cluster(b);
          else ptx::mbar_arrive(b);
        }
        pend_mask |= 1u << slot;
        pend_par = (pend_par & ~(1u << slot)) | (phase << slot);
        if (++slot == k4ScaleSlots) {
          slot = 0;
          phase ^= 1;
        }
      }
    }
    // every commit on a slot's barrier has arrived before the CTA leaves
    volatile int no_abort = 0;
    for (int s = 0; s < k4ScaleSlots; ++s) {
      if ((pend_mask & (1u << s)) && !*abort_flag)
        ptx::mbar_wait_bounded(ptx::smem_addr(&sh.sempty[s]), (pend_par >> s) & 1u, &no_abort, kDrainNs);
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
