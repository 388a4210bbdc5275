// gemm_w8a8.cu -- the 8-bit product with a scale for each token and each output channel, for
// batches of few tokens, on sm_100a (tcgen05 kind::i8).
//
//   acc[t, o] = sum_j Xq[t, j] Wq[o, j]  (int32, exact),
//   Y[t, o] = T_rn(fl32(fl32(fl32(acc) fl32(amax_t / 127)) fl32(wmax_o / 127))).
// Sparse-BitNet summary ("Sparse-BitNet：1.58-bit 大模型天然兼容半结构化稀疏"), 前置知识: activations are
// absmax-quantised to 8 bits per token; here the weight rows are too (both by sbl_act_quant), for
// the projections that are not ternary.
//
// With few tokens the product is bound by reading Wq once.  The weight rows are the M = 128
// operand and the tokens the N operand (16 .. 256), so a short batch wastes no weight bandwidth;
// the K range of a 128-row tile is split over a cluster of blocks so that every SM streams
// weights, each through its own TMA ring.  The blocks of a cluster then exchange their int32
// partial tiles through distributed shared memory: block r adds up the token columns r, r + CS, ...
// of all of them.  int32 sums are exact in any order.  A warp writes 32 neighbouring outputs of a
// token.  Barriers, tensor memory and descriptors are set up while the previous kernel finishes
// (programmatic dependent launch); global memory is touched only after it has.
// Every mbarrier wait is bounded (sbl_device.cuh).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "block_norm.cuh"
#include "sbl_device.cuh"
#include "sbl_internal.h"

namespace sbl {
namespace {

constexpr int kW8Rows = 128;     // weight rows per tile
constexpr int kW8Threads = 192;  // producer warp, MMA warp, 4 epilogue warps

struct W8Args {
  const float* amax;
  const float* wmax;
  void* Y;
  int T, d_out, KB;  // KB: 128-byte blocks of K
  int mt;            // weight row tiles
  uint32_t* err;
};

template <int BN, int STAGES>
struct W8Cfg {
  static constexpr int A_BYTES = kW8Rows * 128;
  static constexpr int B_BYTES = BN * 128;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int PART_BYTES = BN * kW8Rows * 4;  // a block's partial tile, over the ring
  static constexpr int RING_BYTES = STAGES * STAGE_BYTES > PART_BYTES ? STAGES * STAGE_BYTES : PART_BYTES;
  static constexpr int SMEM_BYTES = RING_BYTES + 1024 /*align*/ + BN * 4 + 256;
  static constexpr uint32_t TMEM_COLS = BN < 32 ? 32 : BN;
  static constexpr uint32_t IDESC = instr_desc(true, kW8Rows, BN, false, false);
};

template <bool kBf16>
__device__ __forceinline__ void w8_store(void* Y, long long at, int acc, float sx, float sw) {
  const float y = __fmul_rn(__fmul_rn(__int2float_rn(acc), sx), sw);
  if constexpr (kBf16)
    static_cast<__nv_bfloat16*>(Y)[at] = __float2bfloat16_rn(y);
  else
    static_cast<float*>(Y)[at] = y;
}

template <int BN, int STAGES, bool kBf16>
__global__ void __launch_bounds__(kW8Threads) w8a8_stream_kernel(const __grid_constant__ CUtensorMap tmW,
                                                                 const __grid_constant__ CUtensorMap tmX,
                                                                 const W8Args a) {
  using C = W8Cfg<BN, STAGES>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* s_sx = reinterpret_cast<float*>(smem + C::RING_BYTES);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::RING_BYTES + BN * 4);
  uint64_t* empty = full + STAGES;
  uint64_t* done = empty + STAGES;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  uint32_t cs, rank;
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(cs));
  rank = pair::cluster_rank();
  const int tile = static_cast<int>(blockIdx.x / cs);
  const int m0 = (tile % a.mt) * kW8Rows;
  const int n0 = (tile / a.mt) * BN;
  const int kb0 = static_cast<int>(static_cast<long long>(a.KB) * rank / cs);
  const int kb1 = static_cast<int>(static_cast<long long>(a.KB) * (rank + 1) / cs);

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmX);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // after the allocation: a successor that starts early cannot take the columns this block needs
  asm volatile("griddepcontrol.launch_dependents;");

  if (warp == 0) {
    if (lane == 0) {
      pdl::wait();
      int it = 0;
      bool ok = true;
      for (int kb = kb0; kb < kb1; ++kb, ++it) {
        const int s = it % STAGES;
        if (!mbar_wait(&empty[s], (static_cast<uint32_t>(it / STAGES) & 1u) ^ 1u, abort_flag, a.err)) {
          ok = false;
          break;
        }
        mbar_arrive_expect_tx(&full[s], C::STAGE_BYTES);
        tma_load_2d(smem + s * C::STAGE_BYTES, &tmW, &full[s], kb * 128, m0);
        tma_load_2d(smem + s * C::STAGE_BYTES + C::A_BYTES, &tmX, &full[s], kb * 128, n0);
      }
      if (!ok) {  // let the copies in flight land before the block exits
        for (int i = (it > STAGES ? it - STAGES : 0); i < it; ++i)
          mbar_wait(&full[i % STAGES], static_cast<uint32_t>(i / STAGES) & 1u, nullptr, a.err);
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      int it = 0;
      for (int kb = kb0; kb < kb1; ++kb, ++it) {
        const int s = it % STAGES;
        if (!mbar_wait(&full[s], static_cast<uint32_t>(it / STAGES) & 1u, abort_flag, a.err)) break;
        tc_fence_after();
        const uint32_t sa = smem_u32(smem + s * C::STAGE_BYTES);
        const uint32_t sb = sa + C::A_BYTES;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma<true>(tmem, smem_desc_sw128(sa + kk * 32, 16, 1024), smem_desc_sw128(sb + kk * 32, 16, 1024), C::IDESC,
                     (kb > kb0 || kk > 0) ? 1u : 0u);
        umma_commit(&empty[s]);
      }
      umma_commit(done);  // fires when this block's MMAs are complete (also after giving up)
    }
  } else {
    const int q = warp & 3;  // TMEM lane quarter this warp may read
    const int row = 32 * q + lane;
    const int o = m0 + row;
    pdl::wait();
    for (int c = threadIdx.x - 64; c < BN; c += 128)
      s_sx[c] = n0 + c < a.T ? __fdiv_rn(a.amax[n0 + c], 127.0f) : 0.0f;
    const float sw = o < a.d_out ? __fdiv_rn(a.wmax[o], 127.0f) : 0.0f;
    asm volatile("bar.sync 1, 128;" ::: "memory");
    const int cols = min(BN, a.T - n0);
    mbar_wait(done, 0, abort_flag, a.err);
    tc_fence_after();
    int32_t* part = reinterpret_cast<int32_t*>(smem);  // [BN][128], over the ring: all MMAs have read it
    const uint32_t tbase = tmem + (static_cast<uint32_t>(32 * q) << 16);
#pragma unroll 1
    for (int c0 = 0; c0 < cols; c0 += 32) {
      uint32_t r[32];
      tmem_ld_32x32b_x32(tbase + static_cast<uint32_t>(c0), r);
      tmem_ld_wait();
      if (cs == 1) {
        if (o < a.d_out) {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (c0 + j < cols)
              w8_store<kBf16>(a.Y, static_cast<long long>(n0 + c0 + j) * a.d_out + o, static_cast<int>(r[j]),
                              s_sx[c0 + j], sw);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (c0 + j < cols) part[(c0 + j) * kW8Rows + row] = static_cast<int>(r[j]);
      }
    }
  }
  if (cs > 1) {
    __syncwarp();
    pair::cluster_sync();  // every block's partial tile is in its shared memory
    if (warp >= 2) {
      const int row = 32 * (warp & 3) + lane;
      const int o = m0 + row;
      const int cols = min(BN, a.T - n0);
      const float sw = o < a.d_out ? __fdiv_rn(a.wmax[o], 127.0f) : 0.0f;
      const uint32_t base = smem_u32(smem) + static_cast<uint32_t>(row) * 4u;
      // eight columns at a time from every block: up to 64 remote loads in flight
      for (int c0 = static_cast<int>(rank); c0 < cols; c0 += 8 * static_cast<int>(cs)) {
        int acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
        for (uint32_t p = 0; p < 8; ++p) {
          if (p >= cs) break;
          const uint32_t from = pair::map_to(base, p);
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const int c = c0 + u * static_cast<int>(cs);
            int v = 0;
            if (c < cols)
              asm volatile("ld.shared::cluster.s32 %0, [%1];"
                           : "=r"(v)
                           : "r"(from + static_cast<uint32_t>(c) * (kW8Rows * 4u))
                           : "memory");
            acc[u] += v;
          }
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int c = c0 + u * static_cast<int>(cs);
          if (c < cols && o < a.d_out)
            w8_store<kBf16>(a.Y, static_cast<long long>(n0 + c) * a.d_out + o, acc[u], s_sx[c], sw);
        }
      }
    }
    __syncwarp();
    pair::cluster_sync();  // no block leaves while its partial tile is being read
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

template <int BN, int STAGES, bool kBf16>
cudaError_t run(const int8_t* Xq, const int8_t* Wq, int d_in, W8Args a, int blocks_per_sm, cudaStream_t stream,
                int num_sms) {
  using C = W8Cfg<BN, STAGES>;
  CUtensorMap tw, tx;
  if (!make_tmap_u8(&tw, Wq, d_in, a.d_out, d_in, 128, kW8Rows, true) ||
      !make_tmap_u8(&tx, Xq, d_in, a.T, d_in, 128, BN, true))
    return cudaErrorInvalidValue;
  auto kern = w8a8_stream_kernel<BN, STAGES, kBf16>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
  if (e != cudaSuccess) return e;
  const int tiles = a.mt * ((a.T + BN - 1) / BN);
  // as many K splits as keep the whole grid resident, at least two K blocks each
  int cs = 8;
  while (cs > 1 && (static_cast<long long>(tiles) * cs > static_cast<long long>(num_sms) * blocks_per_sm ||
                    a.KB < 2 * cs))
    --cs;
  return pdl::launch(kern, tiles * cs, kW8Threads, C::SMEM_BYTES, cs, stream, tw, tx, a);
}

template <bool kBf16>
cudaError_t dispatch(const int8_t* Xq, const int8_t* Wq, int d_in, const W8Args& a, cudaStream_t stream, int num_sms) {
  if (a.T <= 16) return run<16, 6, kBf16>(Xq, Wq, d_in, a, 2, stream, num_sms);
  if (a.T <= 32) return run<32, 5, kBf16>(Xq, Wq, d_in, a, 2, stream, num_sms);
  if (a.T <= 64) return run<64, 4, kBf16>(Xq, Wq, d_in, a, 2, stream, num_sms);
  if (a.T <= 128) return run<128, 3, kBf16>(Xq, Wq, d_in, a, 2, stream, num_sms);
  return run<256, 4, kBf16>(Xq, Wq, d_in, a, 1, stream, num_sms);
}

}  // namespace

cudaError_t launch_w8a8(const int8_t* Xq, const float* amax, const int8_t* Wq, const float* wmax, int T, int d_in,
                        int d_out, bool y_bf16, void* Y, cudaStream_t stream, int num_sms, uint32_t* err) {
  // The CTA-pair kernel wins once its 256 x 256 tiles fill the device.
  const long long pair_tiles = static_cast<long long>((T + 255) / 256) * ((d_out + 255) / 256);
  if (pair_tiles >= num_sms / 2)
    return launch_forward_w8a8_pair(Xq, amax, Wq, wmax, T, d_in, d_out, y_bf16, Y, stream, num_sms, err);
  W8Args a{};
  a.amax = amax;
  a.wmax = wmax;
  a.Y = Y;
  a.T = T;
  a.d_out = d_out;
  a.KB = (d_in + 127) / 128;
  a.mt = (d_out + kW8Rows - 1) / kW8Rows;
  a.err = err;
  return y_bf16 ? dispatch<true>(Xq, Wq, d_in, a, stream, num_sms)
                : dispatch<false>(Xq, Wq, d_in, a, stream, num_sms);
}

}  // namespace sbl
