// block_norm.cuh -- what the block norm's forward and backward kernels share: 4 neighbouring
// columns in either type, and the ring of rows that bulk copies keep ahead of the arithmetic.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "pdl.cuh"
#include "sbl_device.cuh"

namespace sbl {

// Two fp32 operations per instruction (sm_100), each rounded as the single one.  The compiler fuses a
// packed product with a packed sum, whatever rounding they name (measured: h' then differs in its
// last bit), so a sum that has to see the rounded product is written with the single instructions.
__device__ __forceinline__ float2 splat2(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 mul2(const float2& a, const float2& b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 add2(const float2& a, const float2& b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 fma2(const float2& a, const float2& b, const float2& c) {
  return __ffma2_rn(a, b, c);
}

__device__ __forceinline__ float2 unpack2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// one packed conversion (round to nearest even)
__device__ __forceinline__ uint32_t pack2(const float2& x) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(x.x, x.y);
  return *reinterpret_cast<const uint32_t*>(&p);
}

// Columns 4 i .. 4 i + 3 of a staged row, bf16 (kBf16) or fp32, as two pairs.
template <bool kBf16>
__device__ __forceinline__ void staged22(const uint8_t* row, int i, float2 (&x)[2]) {
  if constexpr (kBf16) {
    const uint2 w = reinterpret_cast<const uint2*>(row)[i];
    x[0] = unpack2(w.x);
    x[1] = unpack2(w.y);
  } else {
    const float4 v = reinterpret_cast<const float4*>(row)[i];
    x[0] = make_float2(v.x, v.y);
    x[1] = make_float2(v.z, v.w);
  }
}

// Bulk copy of `bytes` (a multiple of 16) from global memory to shared memory, both 16-byte
// aligned; completes on `bar`.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// Position in a ring of `depth` slots, with the parity of the barrier phase that fills it.
struct RingPos {
  int slot = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next(int depth) {
    if (++slot == depth) {
      slot = 0;
      parity ^= 1u;
    }
  }
};

// Barrier of the TPR threads of row lane `rib` (within a warp, or one named barrier per lane), so
// the lanes of a block keep their own pace.  A slot may be refilled behind it: every value read from
// the slot has gone into the sums that the threads bring to the barrier.
template <int TPR, int THREADS>
__device__ __forceinline__ void lane_sync(int rib) {
  if constexpr (TPR <= 32)
    __syncwarp();
  else if constexpr (TPR == THREADS)
    __syncthreads();
  else
    asm volatile("bar.sync %0, %1;" ::"r"(rib + 1), "n"(TPR) : "memory");
}

}  // namespace sbl
