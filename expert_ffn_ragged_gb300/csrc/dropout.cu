// dropout.cu -- dropout by a counter-based generator, with the residual added (rd_dropout_rows).
//
// A stream: x, residual and out cross HBM once and the mask never does.  One call of the generator (Philox
// 4x32, ten rounds of two 32 x 32 -> 64 bit products; J. Salmon et al., 2011) gives 128 bits, 16 for each of the
// eight elements of a vector: with 32 bits an element the products would cost as much time as
// the bytes.  Each element's draw depends on its place alone, so the gradient's call draws the same.
// Bound: HBM.  28157 x 4096, bf16 onto an f32 residual: 1.15 GB in 180 us (6.4 TB/s); bf16 without a residual 461 MB in 81 us,
// where the generator's products (some 70 of 100 instructions a vector) count too.  16 x 4096: 2.0 us, a launch.
#include <cuda_runtime.h>
#include <stdint.h>

#include "block_args.h"
#include "launch.h"
#include "rows.cuh"

namespace rd {
namespace {

__device__ __forceinline__ void philox_round(uint32_t (&c)[4], uint32_t k0, uint32_t k1) {
  const uint64_t a = static_cast<uint64_t>(0xD2511F53u) * c[0], b = static_cast<uint64_t>(0xCD9E8D57u) * c[2];
  const uint32_t c1 = c[1], c3 = c[3];
  c[0] = static_cast<uint32_t>(b >> 32) ^ c1 ^ k0;
  c[1] = static_cast<uint32_t>(b);
  c[2] = static_cast<uint32_t>(a >> 32) ^ c3 ^ k1;
  c[3] = static_cast<uint32_t>(a);
}

__device__ __forceinline__ void philox(uint64_t counter, uint64_t offset, uint64_t key, uint32_t (&c)[4]) {
  c[0] = static_cast<uint32_t>(counter);
  c[1] = static_cast<uint32_t>(counter >> 32);
  c[2] = static_cast<uint32_t>(offset);
  c[3] = static_cast<uint32_t>(offset >> 32);
  uint32_t k0 = static_cast<uint32_t>(key), k1 = static_cast<uint32_t>(key >> 32);
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    philox_round(c, k0, k1);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
}

constexpr int kDropThreads = 256;
constexpr int kDropBatch = 2;  // vectors of a thread in flight

template <class X, class O, bool RES>
__global__ void __launch_bounds__(kDropThreads) dropout_rows_kernel(const DropoutArgs a) {
  pdl_trigger();
  pdl_wait();
  const int64_t total = static_cast<int64_t>(rows_within(a.limit, a.rows)) * a.vecs;
  const uint64_t key = static_cast<uint64_t>(a.rng[0]), offset = static_cast<uint64_t>(a.rng[1]);
  const X* x = static_cast<const X*>(a.x);
  const O* res = static_cast<const O*>(a.residual);
  O* out = static_cast<O*>(a.out);
  const uint32_t least = static_cast<uint32_t>(a.least);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kDropThreads * kDropBatch;
  for (int64_t v0 = static_cast<int64_t>(blockIdx.x) * kDropThreads * kDropBatch + threadIdx.x; v0 < total;
       v0 += step) {
    Raw8<X> rx[kDropBatch];
    Raw8<O> rr[kDropBatch];
#pragma unroll
    for (int i = 0; i < kDropBatch; ++i) {
      const int64_t v = v0 + i * kDropThreads;
      if (v < total) {
        load_raw(rx[i], x + 8 * v);
        if (RES) load_raw(rr[i], res + 8 * v);
      }
    }
#pragma unroll
    for (int i = 0; i < kDropBatch; ++i) {
      const int64_t v = v0 + i * kDropThreads;
      if (v >= total) continue;
      uint32_t words[4];
      philox(static_cast<uint64_t>(v), offset, key, words);
      float e[8], r[8];
      widen(rx[i], e);
      if (RES) widen(rr[i], r);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t draw = (j & 1) ? words[j >> 1] >> 16 : words[j >> 1] & 0xFFFFu;
        e[j] = draw >= least ? e[j] * a.scale : 0.0f;
        if (RES) e[j] += r[j];
      }
      store8(out + 8 * v, e);
    }
  }
}

// Six blocks an SM with two vectors a thread (us on 3 / 4 / 6 / 8 blocks: f32 residual 197 / 186 / 183 / 184, bf16 residual 119 / 114 /
// 114 / 129, none 94 / 87 / 81 / 79).
template <class X, class O>
cudaError_t go(const DropoutArgs& a, int sms, cudaStream_t stream) {
  const int64_t per = kDropThreads * kDropBatch;
  const int64_t blocks = (static_cast<int64_t>(a.rows) * a.vecs + per - 1) / per, most = static_cast<int64_t>(sms) * 6;
  const dim3 grid(static_cast<unsigned>(blocks < most ? blocks : most));
  return a.residual != nullptr ? launch_pdl(dropout_rows_kernel<X, O, true>, grid, kDropThreads, 0, 1, stream, a)
                               : launch_pdl(dropout_rows_kernel<X, O, false>, grid, kDropThreads, 0, 1, stream, a);
}

}  // namespace

cudaError_t launch_dropout_rows(const DropoutArgs& a, int dtype, int out_dtype, int sms,
                                cudaStream_t stream) {
  if (dtype == RD_F32)
    return out_dtype == RD_F32 ? go<float, float>(a, sms, stream) : go<float, bf16>(a, sms, stream);
  return out_dtype == RD_F32 ? go<bf16, float>(a, sms, stream) : go<bf16, bf16>(a, sms, stream);
}

}  // namespace rd
