// launch.h -- launches that may begin before the kernel in front of them on the stream has ended.
//
// The kernels of rd_moe.h follow one another in a layer, several of them a few microseconds long, so
// the gap between two launches is a good part of their time.  They are launched with programmatic
// stream serialisation: a kernel's blocks may start, and set up what needs no memory of the stream's
// earlier work, while the previous kernel still runs.  pdl_wait() comes before the first access to
// global memory in every block of every such kernel and returns when all earlier work of the stream
// is complete and visible; pdl_trigger() lets the next launch begin once every block has come to it.
// The kernels read with plain loads: what the previous kernel writes is not read-only for the lifetime of a
// kernel that starts before its end, as the non-coherent path and restrict would have it.
// Measured, one pass after another: route 32771 x 256 and 4-bit rows there and back each lose one gap
// of about 2 us between their two kernels.
#pragma once

#include <cuda_runtime.h>

namespace rd {

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// one launch of `kernel`; cluster > 1: clusters of that many blocks along x
template <class... Params, class... Args>
cudaError_t launch_pdl(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, int cluster,
                       cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

}  // namespace rd
