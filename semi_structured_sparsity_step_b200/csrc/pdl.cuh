// pdl.cuh -- programmatic dependent launch, as the block norm, the 8-bit product and the gradient
// group use it.
#pragma once

#include <cuda_runtime.h>
#include <cstdint>

namespace sbl {

// Programmatic dependent launch: a kernel may be set up while the previous one of its stream
// finishes, and touches global memory only after wait().  Loads behind it are ordinary ones: memory that the
// previous kernel writes is not constant for this kernel's life, as a read-only load (__ldg) asks for
// and a __restrict__ pointer lets the compiler assume, which could then move it ahead of wait().
namespace pdl {

__device__ __forceinline__ void wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Load that stays behind wait(), by its place among volatile statements, and that the compiler may still take
// ahead of the kernel's own stores: a plain one could alias them.
__device__ __forceinline__ uint2 load(const uint2* p) {
  uint2 v;
  asm volatile("ld.global.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}
__device__ __forceinline__ uint4 load(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// The next kernel may be set up once every block has called this or ended.  Called behind wait(), so that
// a kernel that reads ahead of its own wait (the decode GEMVs read packed weights) finds whole what
// the kernels before this one wrote.
__device__ __forceinline__ void release() { asm volatile("griddepcontrol.launch_dependents;"); }

template <typename... KArgs, typename... Args>
cudaError_t launch(void (*kern)(KArgs...), int grid, int threads, int smem, int cluster, cudaStream_t stream,
                   Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
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
  return cudaLaunchKernelEx(&cfg, kern, static_cast<Args&&>(args)...);
}

}  // namespace pdl

}  // namespace sbl
