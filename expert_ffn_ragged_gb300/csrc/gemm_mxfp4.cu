// gemm_mxfp4.cu -- launches of the grouped product over 4-bit operands.
#include "gemm_mxfp4.cuh"

namespace rd {
namespace {

template <int EPI, int VAR>
cudaError_t launch_impl(const Gemm4Maps& maps, const Gemm4Args& args, int grid, cudaStream_t stream) {
  constexpr bool PAIR = VAR == k4Pair;
  constexpr size_t smem = gemm4_smem_bytes<VAR>();
  static_assert(smem <= 232448, "shared memory of one CTA");
  const auto kernel = grouped_gemm_mxfp4_kernel<EPI, VAR>;
  static std::atomic<bool> attr_set[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[dev].load(std::memory_order_acquire)) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    attr_set[dev].store(true, std::memory_order_release);
  }
  if (PAIR) {
    // as for the bf16 products: no more CTA pairs than can be resident at once
    static std::atomic<int> max_clusters[64];
    int clusters = max_clusters[dev].load(std::memory_order_acquire);
    if (clusters == 0) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
      cfg.blockDim = dim3(k4Threads, 1, 1);
      cfg.dynamicSmemBytes = smem;
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = 2;
      attr[0].val.clusterDim.y = 1;
      attr[0].val.clusterDim.z = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      int n = 0;
      const cudaError_t e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
      if (e != cudaSuccess) return e;
      clusters = n > 0 ? n : 1;
      max_clusters[dev].store(clusters, std::memory_order_release);
    }
    if (grid > 2 * clusters) grid = 2 * clusters;
  }
  return launch_pdl(kernel, dim3(static_cast<unsigned>(grid)), k4Threads, smem, PAIR ? 2 : 1, stream, maps,
                    args);
}

template <int VAR>
cudaError_t launch_epi(int epi, const Gemm4Maps& maps, const Gemm4Args& args, int grid,
                       cudaStream_t stream) {
  switch (epi) {
    case k4EpiNone: return launch_impl<k4EpiNone, VAR>(maps, args, grid, stream);
    case k4EpiGlu: return launch_impl<k4EpiGlu, VAR>(maps, args, grid, stream);
    default: return launch_impl<k4EpiGluQuant, VAR>(maps, args, grid, stream);
  }
}

}  // namespace

cudaError_t launch_gemm_mxfp4(int epi, int variant, const Gemm4Maps& maps, const Gemm4Args& args,
                              int grid, cudaStream_t stream) {
  switch (variant) {
    case k4Pair: return launch_epi<k4Pair>(epi, maps, args, grid, stream);
    case k4Single: return launch_epi<k4Single>(epi, maps, args, grid, stream);
    default: return launch_epi<k4Few>(epi, maps, args, grid, stream);
  }
}

}  // namespace rd
