// gemm_linear.cu -- the forward grouped GEMM with bias, activation and residual in its epilogue
// (rd_linear), bf16 and f32 outputs, single-CTA and CTA-pair variants.
#include "gemm_kernel.cuh"

namespace rd {
cudaError_t launch_gemm_linear(bool f32_out, bool pair, const CUtensorMap& a, const CUtensorMap& b,
                               const GemmArgs& args, int grid, cudaStream_t s) {
  if (pair)
    return f32_out ? launch_gemm_impl<kOpFwd, kEpiLinearF32, true>(a, b, args, grid, s)
                   : launch_gemm_impl<kOpFwd, kEpiLinear, true>(a, b, args, grid, s);
  return f32_out ? launch_gemm_impl<kOpFwd, kEpiLinearF32, false>(a, b, args, grid, s)
                 : launch_gemm_impl<kOpFwd, kEpiLinear, false>(a, b, args, grid, s);
}
}  // namespace rd
