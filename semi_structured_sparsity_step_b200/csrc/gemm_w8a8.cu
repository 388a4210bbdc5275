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
// weights, each through its own TMA ring.  The blocks of a cluster then add their int32 partial
// tiles up through distributed shared memory, each block a share of the token columns, by bulk
// reductions into its shared memory (reading the other blocks' tiles word by word instead pays their
// latency over and over: 28 us against 8 at 256 x 2048 x 2048 in four splits).  int32 sums are exact
// in any order.  A warp writes 32 neighbouring outputs of a token.  Barriers, tensor memory and
// descriptors are set up while the previous kernel finishes (programmatic dependent launch); global
// memory is touched only after it has.
// Every mbarrier wait is bounded (sbl_device.cuh).
//
// Measured: 1 x 11008 x 32768 (361 MB of weights) 55.6 us, the measured copy rate; 1 x 2048 x 11008
// 6.4 us and 509 x 2048 x 2048 7.4 us with the operands in L2, of which about 3 us are the launch and
// the first copy's latency.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cmath>
#include <cstdint>

#include "pdl.cuh"
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
  int nt;            // token tiles
  uint32_t* err;
};

template <int BN, int STAGES>
struct W8Cfg {
  static constexpr int A_BYTES = kW8Rows * 128;
  static constexpr int B_BYTES = BN * 128;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int PART_BYTES = BN * kW8Rows * 4;  // a block's partial tile, over the ring
  static constexpr int RING_BYTES = STAGES * STAGE_BYTES > PART_BYTES ? STAGES * STAGE_BYTES : PART_BYTES;
  static constexpr int SX = BN < 32 ? 32 : BN;  // token scales (read 32 at a time)
  static constexpr int SMEM_BYTES = RING_BYTES + 1024 /*align*/ + SX * 4 + 256;
  static constexpr uint32_t TMEM_COLS = BN < 32 ? 32 : BN;
  static constexpr uint32_t IDESC = instr_desc(true, kW8Rows, BN, false, false);
};

__device__ __forceinline__ float w8_scaled(int acc, float sx, float sw) {
  return __fmul_rn(__fmul_rn(__int2float_rn(acc), sx), sw);
}

template <bool kBf16>
__device__ __forceinline__ void w8_store(void* Y, long long at, float y) {
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
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::RING_BYTES + C::SX * 4);
  uint64_t* empty = full + STAGES;
  uint64_t* done = empty + STAGES;
  uint64_t* joined = done + 1;  // the other blocks' partial sums have arrived
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(joined + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  uint32_t cs, rank;
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(cs));
  rank = pair::cluster_rank();
  const int tile = static_cast<int>(blockIdx.x / cs);
  // token tiles vary fastest: the blocks that read the same weight rows run together, and Wq comes from
  // HBM once
  const int m0 = (tile / a.nt) * kW8Rows;
  const int n0 = (tile % a.nt) * BN;
  const int kb0 = static_cast<int>(static_cast<long long>(a.KB) * rank / cs);
  const int kb1 = static_cast<int>(static_cast<long long>(a.KB) * (rank + 1) / cs);

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(done, 1);
    mbar_init(joined, 1);
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
  if (warp == 0) {
    if (lane == 0) {
      pdl::wait();
      pdl::release();  // this block has its tensor memory
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
    for (int c = threadIdx.x - 64; c < C::SX; c += 128)
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
      tmem_ld_wait_for(r);
      if (cs == 1) {
        // every result before the first store: a store could alias the scales for all the compiler
        // knows, and each scale would wait for the store before it (65 cycles a column, measured)
        float y[32];
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          const float4 sx = *reinterpret_cast<const float4*>(s_sx + c0 + j);
          y[j] = w8_scaled(static_cast<int>(r[j]), sx.x, sw);
          y[j + 1] = w8_scaled(static_cast<int>(r[j + 1]), sx.y, sw);
          y[j + 2] = w8_scaled(static_cast<int>(r[j + 2]), sx.z, sw);
          y[j + 3] = w8_scaled(static_cast<int>(r[j + 3]), sx.w, sw);
        }
        if (o < a.d_out) {
          long long at = static_cast<long long>(n0 + c0) * a.d_out + o;
#pragma unroll
          for (int j = 0; j < 32; ++j, at += a.d_out)
            if (c0 + j < cols) w8_store<kBf16>(a.Y, at, y[j]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (c0 + j < cols) part[(c0 + j) * kW8Rows + row] = static_cast<int>(r[j]);
      }
    }
  }
  if (cs > 1) {
    // Block r ends up with the token columns [r share, (r + 1) share): every other block adds its
    // partial sums of them into r's tile, one bulk reduction per pair of blocks.
    const int cols = min(BN, a.T - n0);
    const int share = (cols + static_cast<int>(cs) - 1) / static_cast<int>(cs);
    auto first_of = [&](uint32_t r) { return min(cols, static_cast<int>(r) * share); };
    const int c_lo = first_of(rank), c_hi = first_of(rank + 1);
    if (threadIdx.x == 64) mbar_arrive_expect_tx(joined, static_cast<uint32_t>(c_hi - c_lo) * kW8Rows * 4u * (cs - 1));
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the tile was written by ordinary stores
    __syncwarp();
    pair::cluster_sync();  // every block's partial tile is in its shared memory
    if (threadIdx.x == 64) {
      for (uint32_t d = 1; d < cs; ++d) {
        const uint32_t p = rank + d < cs ? rank + d : rank + d - cs;
        const int lo = first_of(p), n = first_of(p + 1) - lo;
        if (n == 0) continue;
        const uint32_t src = smem_u32(smem) + static_cast<uint32_t>(lo) * (kW8Rows * 4u);
        asm volatile(
            "cp.reduce.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes.add.s32 [%0], [%1], %2, [%3];" ::"r"(
                pair::map_to(src, p)),
            "r"(src), "r"(static_cast<uint32_t>(n) * kW8Rows * 4u), "r"(pair::map_to(smem_u32(joined), p))
            : "memory");
      }
    }
    if (warp >= 2 && c_hi > c_lo) {
      mbar_wait(joined, 0, abort_flag, a.err);
      const int row = 32 * (warp & 3) + lane;
      const int o = m0 + row;
      const float sw = o < a.d_out ? __fdiv_rn(a.wmax[o], 127.0f) : 0.0f;
      const int32_t* part = reinterpret_cast<const int32_t*>(smem) + row;
      for (int c0 = c_lo; c0 < c_hi; c0 += 8) {
        float y[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int c = min(c0 + u, c_hi - 1);
          y[u] = w8_scaled(part[c * kW8Rows], s_sx[c], sw);
        }
        if (o < a.d_out) {
          long long at = static_cast<long long>(n0 + c0) * a.d_out + o;
#pragma unroll
          for (int u = 0; u < 8; ++u, at += a.d_out)
            if (c0 + u < c_hi) w8_store<kBf16>(a.Y, at, y[u]);
        }
      }
    }
    __syncwarp();
    pair::cluster_sync();  // no block leaves while its tile is being added to or read
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

template <int BN, int STAGES, bool kBf16>
cudaError_t run(const int8_t* Xq, const int8_t* Wq, int d_in, W8Args a, int cs, cudaStream_t stream) {
  using C = W8Cfg<BN, STAGES>;
  CUtensorMap tw, tx;
  if (!make_tmap_u8(&tw, Wq, d_in, a.d_out, d_in, 128, kW8Rows, true) ||
      !make_tmap_u8(&tx, Xq, d_in, a.T, d_in, 128, BN, true))
    return cudaErrorInvalidValue;
  auto kern = w8a8_stream_kernel<BN, STAGES, kBf16>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
  if (e != cudaSuccess) return e;
  a.nt = (a.T + BN - 1) / BN;
  const int tiles = (a.d_out + kW8Rows - 1) / kW8Rows * a.nt;
  return pdl::launch(kern, tiles * cs, kW8Threads, C::SMEM_BYTES, cs, stream, tw, tx, a);
}

// Which kernel a product goes to: token tile (0: the CTA-pair kernel) and K splits.
struct W8Plan {
  int bn, cs;
};

// The fastest by a model of the time in ns, fitted to 458 cases (T 1 .. 8192, d_in 128 .. 11008, d_out
// 128 .. 32768, both types), on which the plan it picks is 1.1% above the fastest of all token tiles and
// splits on average, and more than 10% above it in 14 cases (the worst 19%).  It is fitted to order the plans; a
// time that it gives can be further off (422 x 3536 -> 10328, 82 tiles of 256 x 256 on 74 pairs: 19 us given,
// 30 to 33 measured):
//   streaming kernel: 4000 for the launch, plus the longest of
//     what an SM copies from L2 (its blocks x their K blocks x 16 KB + 128 BN) at 186 bytes/ns, 89 with
//     more than one block on it, 168 at BN 256,
//     what all copy together at 18200 bytes/ns, and
//     Wq from HBM at 5500 bytes/ns or 54 per block of the last wave, half more for each further token tile,
//   plus the end of a block, once per wave: 540 + 21.3 per token column (14.1 of fp32), or 1230 + 19.3
//   with a cluster's exchange (and then one wave at most);
//   CTA-pair kernel: 7700, plus the longer of both operands from HBM at 4800 bytes/ns and, for each wave
//   of 256 x 256 tiles, the longer of 205 per K block and the 1550 (fp32 3200) of a tile's epilogue.
// The constants are those of the best fit, where a choice depends on differences, not rates of the machine.
// Measured, best plan against one fixed choice (token tile >= T, as many splits as fit):
// 512 x 2048 x 2048 7.6 us against 12.4, 256 x 2048 x 2048 7.5 against 19.9, 1 x 2048 x 32768 13.7
// against 22.5 on CTA pairs, 2048 x 896 x 4864 17.0 on CTA pairs against 20.5.
W8Plan plan_w8a8(int T, int d_in, int d_out, bool y_bf16, int num_sms) {
  const double KB = (d_in + 127) / 128, mt = (d_out + kW8Rows - 1) / kW8Rows;
  const double pair_tiles = static_cast<double>((T + 255) / 256) * ((d_out + 255) / 256);
  const double pairs = num_sms / 2;
  const double pair_end = y_bf16 ? 1550.0 : 3200.0;
  const double pair_wave = KB * 205.0 > pair_end ? KB * 205.0 : pair_end;
  const double pair_math = static_cast<double>(static_cast<long long>((pair_tiles + pairs - 1) / pairs)) * pair_wave;
  const double pair_hbm = (static_cast<double>(d_out) + T) * d_in / 4800.0;
  double best = 7700.0 + (pair_math > pair_hbm ? pair_math : pair_hbm);
  W8Plan plan{0, 1};
  for (int bn = 16; bn <= 256; bn *= 2) {
    const double nt = (T + bn - 1) / bn;
    for (int cs = 1; cs <= 8 && (cs == 1 || 2 * cs <= KB); ++cs) {
      const double blocks = mt * nt * cs;
      const double per_sm = static_cast<double>(static_cast<long long>((blocks + num_sms - 1) / num_sms));
      const double kb = static_cast<double>(static_cast<long long>((KB + cs - 1) / cs));
      const double block_bytes = kb * (16384.0 + 128.0 * bn);
      const double copy = per_sm * block_bytes / (bn == 256 ? 168.0 : per_sm > 1 ? 89.0 : 186.0);
      const double copy_all = blocks * block_bytes / 18200.0;
      // clusters do not pack every SM: 254 of 296 places are counted on (288 were measured to take two waves)
      const double resident = num_sms * (bn == 256 ? 1.0 : 2.0) * (cs == 1 ? 1.0 : bn == 256 ? 0.97 : 0.86);
      const double waves = std::ceil(blocks / resident);
      const double last = (blocks - (waves - 1) * resident) / blocks;  // the last wave's share of the blocks
      const double wq = static_cast<double>(d_out) * d_in * (1.0 + 0.5 * (nt - 1));
      const double last_rate = last * blocks * 54.0 < 5500.0 ? last * blocks * 54.0 : 5500.0;
      const double hbm = wq * (1.0 - last) / 5500.0 + wq * last / last_rate;
      const double move = copy > copy_all ? copy : copy_all;
      const double t = 4000.0 + (move > hbm ? move : hbm) +
                       waves * (cs > 1 ? 1230.0 + 19.3 * bn : 540.0 + (y_bf16 ? 21.3 : 14.1) * bn);
      if ((cs == 1 || waves == 1) && t < best) {
        best = t;
        plan = W8Plan{bn, cs};
      }
    }
    if (bn >= T) break;  // a wider tile only adds empty columns
  }
  return plan;
}

template <bool kBf16>
cudaError_t dispatch(const int8_t* Xq, const int8_t* Wq, int d_in, const W8Args& a, const W8Plan& p,
                     cudaStream_t stream) {
  switch (p.bn) {
    case 16: return run<16, 6, kBf16>(Xq, Wq, d_in, a, p.cs, stream);
    case 32: return run<32, 5, kBf16>(Xq, Wq, d_in, a, p.cs, stream);
    case 64: return run<64, 4, kBf16>(Xq, Wq, d_in, a, p.cs, stream);
    case 128: return run<128, 3, kBf16>(Xq, Wq, d_in, a, p.cs, stream);
    default: return run<256, 4, kBf16>(Xq, Wq, d_in, a, p.cs, stream);
  }
}

}  // namespace

cudaError_t launch_w8a8(const int8_t* Xq, const float* amax, const int8_t* Wq, const float* wmax, int T, int d_in,
                        int d_out, bool y_bf16, void* Y, cudaStream_t stream, int num_sms, uint32_t* err) {
  const W8Plan p = plan_w8a8(T, d_in, d_out, y_bf16, num_sms);
  if (p.bn == 0)
    return launch_forward_w8a8_pair(Xq, amax, Wq, wmax, T, d_in, d_out, y_bf16, Y, stream, num_sms, err);
  W8Args a{};
  a.amax = amax;
  a.wmax = wmax;
  a.Y = Y;
  a.T = T;
  a.d_out = d_out;
  a.KB = (d_in + 127) / 128;
  a.err = err;
  return y_bf16 ? dispatch<true>(Xq, Wq, d_in, a, p, stream) : dispatch<false>(Xq, Wq, d_in, a, p, stream);
}

}  // namespace sbl
