// block_norm.cuh -- what the block norm's forward and backward kernels share: loads and stores
// of 4 neighbouring columns in either type, and the dependent launch.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cstdint>

namespace sbl {

__device__ __forceinline__ void unpack4(const uint2& w, float (&x)[4]) {
  x[0] = __uint_as_float(w.x << 16);
  x[1] = __uint_as_float(w.x & 0xFFFF0000u);
  x[2] = __uint_as_float(w.y << 16);
  x[3] = __uint_as_float(w.y & 0xFFFF0000u);
}

// one packed conversion (round to nearest even) per pair
__device__ __forceinline__ uint2 pack4(const float (&x)[4]) {
  const __nv_bfloat162 lo = __floats2bfloat162_rn(x[0], x[1]);
  const __nv_bfloat162 hi = __floats2bfloat162_rn(x[2], x[3]);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
}

// Columns 4 i .. 4 i + 3 of a bf16 (kBf16) or fp32 array (plain loads: the
// output may be the input's own buffer).
template <bool kBf16>
__device__ __forceinline__ void load4(const void* p, long long i, float (&x)[4]) {
  if constexpr (kBf16) {
    unpack4(static_cast<const uint2*>(p)[i], x);
  } else {
    const float4 v = static_cast<const float4*>(p)[i];
    x[0] = v.x;
    x[1] = v.y;
    x[2] = v.z;
    x[3] = v.w;
  }
}

template <bool kBf16>
__device__ __forceinline__ void store4(void* p, long long i, const float (&x)[4]) {
  if constexpr (kBf16) {
    static_cast<uint2*>(p)[i] = pack4(x);
  } else {
    static_cast<float4*>(p)[i] = make_float4(x[0], x[1], x[2], x[3]);
  }
}

// Programmatic dependent launch: a kernel may be set up while the previous one of its stream
// finishes, and touches global memory only after wait().
namespace pdl {

__device__ __forceinline__ void wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

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
