// block_norm.cu -- the seam between two products of a block, forward, in one pass on sm_100a:
// the norm of the branch output, its gate, the scaled residual sum, the next norm and the int8
// quantiser.
//
// Sparse-BitNet summary ("Sparse-BitNet：1.58-bit 大模型天然兼容半结构化稀疏"), Algorithm 1
// step (3): the activation is normalised, then quantised to int8.  With the row y of the branch
// (what the forward product wrote), the residual row h and the token's gate row:
//   r1 = rms(y),  u_j = fl32(fl32(y_j r1) g_post_j)             (u = y without g_post)
//   h'_j = T_rn(fl32(fl32(s h_j) + fl32(gate_j u_j)))           (u_j without a gate)
//   r2 = rms(h'),  xn_j = bf16_rn(fl32(fl32(h'_j r2) g_pre_j)),  then Q_a of the bf16 row xn,
// where rms(x) = fl32(1 / fl32(sqrt(fl32(sum x^2 / d + eps)))) with the sum in fp64, so no summation
// order shows in the int8 codes (norm_quant.cu has the argument).
//
// HBM bound: one read of y and h, one write of h', xn and the codes.  A row lives in registers
// (VPT vectors of 4 columns per thread, TPR threads per row) between its three reductions (sum of
// y^2, sum of h'^2, max |xn|); gains and gate rows come from L1/L2.  The reductions are a chain of
// barriers, so the rows to come are kept on their way: each group of TPR threads has a ring of
// staged rows in shared memory, filled by bulk copies, and refills a slot once its row is in
// registers.  Measured: 32768 x 2048 (y fp32, h bf16, a gate per sequence) 124 us, 0.91 of the measured
// copy rate; one row of 2048 2.4 us, a launch and the chain of three sums.  With 8 columns per thread
// instead of 32 the large case took 185 us: it is the instructions that every thread spends once per
// row that have to be few.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "block_norm.cuh"
#include "sbl_device.cuh"
#include "sbl_internal.h"

namespace sbl {
namespace {

constexpr float kBnMagic = 12582912.0f;  // 1.5 * 2^23: one FADD rounds |t| < 2^22 to an integer

struct BlockNormArgs {
  const void* Y;
  const void* H;
  const uint2* g_post;  // 4 bf16 per vector; NULL: no norm of the branch
  const uint2* gate;    // NULL: no gate
  const uint2* g_pre;
  void* H_out;
  uint2* Xn;      // may be NULL
  uint32_t* Xq;   // 4 codes per vector; may be NULL (then amax is too)
  float* amax;
  float* rstd;    // [2, T]; may be NULL
  float res_scale, eps;
  int period, T, nv;  // nv = d / 4
  int depth;          // rows of the ring
  uint32_t* err;
};

template <int TPR, int THREADS, typename V>
__device__ __forceinline__ V bn_reduce(V x, V* scratch, int rib, bool is_max) {
  constexpr int WPR = TPR < 32 ? 1 : TPR / 32;
#pragma unroll
  for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1) {
    const V y = __shfl_xor_sync(0xFFFFFFFFu, x, o);
    x = is_max ? (x > y ? x : y) : x + y;
  }
  if constexpr (WPR == 1) {
    __syncwarp();
  } else {
    // each reduction of a row has its own scratch, and the barriers of the row's other
    // reductions keep a fast warp from overwriting it before every warp has read it
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = x;
    lane_sync<TPR, THREADS>(rib);
    x = scratch[rib * WPR];
#pragma unroll
    for (int w = 1; w < WPR; ++w) {
      const V y = scratch[rib * WPR + w];
      x = is_max ? (x > y ? x : y) : x + y;
    }
  }
  return x;
}

__device__ __forceinline__ float bn_rstd(double ss, double d, double eps) {
  return __fdiv_rn(1.0f, __fsqrt_rn(static_cast<float>(ss / d + eps)));
}

// int8 code of x in the low byte
__device__ __forceinline__ uint32_t code(float x, float s) {
  return __float_as_uint(__fadd_rn(__fmul_rn(x, s), kBnMagic));
}

// fp64 sum of the squares of a thread's columns, in four chains (one would wait for each addition).
template <int VPT>
__device__ __forceinline__ double sum_squares(const float2 (&x)[VPT][2]) {
  double s[4] = {0.0, 0.0, 0.0, 0.0};
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const double v[4] = {static_cast<double>(x[k][0].x), static_cast<double>(x[k][0].y),
                         static_cast<double>(x[k][1].x), static_cast<double>(x[k][1].y)};
#pragma unroll
    for (int j = 0; j < 4; ++j) s[j] = fma(v[j], v[j], s[j]);
  }
  return (s[0] + s[1]) + (s[2] + s[3]);
}

constexpr int bn_threads(int tpr) { return tpr < 256 ? 256 : tpr; }
// Resident blocks per SM: what the registers of VPT vectors per thread leave room for (one more spills: of
// 6 vectors, 1536 columns, 77 us against 68; of 3 vectors, 384 columns, 80 against 75).
constexpr int bn_blocks(int tpr, int vpt) { return tpr > 256 ? 1 : vpt >= 5 ? 2 : vpt >= 3 ? 3 : 4; }

template <int TPR, int VPT, bool YB, bool HF>
__global__ void __launch_bounds__(bn_threads(TPR), bn_blocks(TPR, VPT)) block_norm_kernel(const BlockNormArgs a) {
  constexpr int THREADS = bn_threads(TPR);
  constexpr int RPB = THREADS / TPR;
  __shared__ double s_y[THREADS / 32], s_h[THREADS / 32];
  __shared__ uint32_t s_max[THREADS / 32];
  const int rib = threadIdx.x / TPR;
  const int tr = threadIdx.x % TPR;
  const double d = static_cast<double>(a.nv) * 4.0;
  const double eps = static_cast<double>(a.eps);
  extern __shared__ __align__(128) uint8_t ring[];
  const uint32_t y_bytes = static_cast<uint32_t>(a.nv) * (YB ? 8u : 16u);
  const uint32_t h_bytes = static_cast<uint32_t>(a.nv) * (HF ? 16u : 8u);
  const uint32_t slot_bytes = y_bytes + h_bytes;
  uint8_t* slots = ring + static_cast<size_t>(rib) * a.depth * slot_bytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(ring + static_cast<size_t>(RPB) * a.depth * slot_bytes) + rib * a.depth;
  const long long stride = static_cast<long long>(gridDim.x) * RPB;
  __shared__ int s_abort;
  if (tr == 0) {
    for (int i = 0; i < a.depth; ++i) mbar_init(&bars[i], 1);
    s_abort = 0;
    fence_mbar_init();
  }
  auto request = [&](long long row, int slot) {
    uint8_t* dst = slots + static_cast<size_t>(slot) * slot_bytes;
    mbar_arrive_expect_tx(&bars[slot], slot_bytes);
    bulk_load(dst, static_cast<const uint8_t*>(a.Y) + row * y_bytes, y_bytes, &bars[slot]);
    bulk_load(dst + y_bytes, static_cast<const uint8_t*>(a.H) + row * h_bytes, h_bytes, &bars[slot]);
  };
  __syncthreads();
  pdl::wait();
  const long long row0 = static_cast<long long>(blockIdx.x) * RPB + rib;
  if (tr == 0)
    for (int i = 0; i < a.depth; ++i)
      if (row0 + i * stride < a.T) request(row0 + i * stride, i);
  // With one row per lane the next kernel is set up meanwhile: 1 x 2048 and the 8-bit product 2048 -> 11008
  // that reads it 7.8 us, without 9.6.  A grid that stays loses: 4096 x 2048 18.4 us against 17.6.
  if (a.T <= stride) pdl::release();

  RingPos pos;
  for (long long base = static_cast<long long>(blockIdx.x) * RPB; base < a.T; base += stride) {
    const long long row = base + rib;
    const bool active = row < a.T;
    const int rc = static_cast<int>(active ? row : static_cast<long long>(a.T) - 1);
    const long long at = static_cast<long long>(rc) * a.nv;
    const uint8_t* staged = slots + static_cast<size_t>(pos.slot) * slot_bytes;
    const int slot = pos.slot;
    if (active) mbar_wait(&bars[slot], pos.parity, &s_abort, a.err);
    pos.next(a.depth);
    float2 y[VPT][2];
    uint2 gain[VPT], gate[VPT];
    // gains and gate row on their way before the sums that their use waits for
    auto fetch = [&](const uint2* p, uint2 (&to)[VPT]) {
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        const int i = tr + k * TPR;
        to[k] = i < a.nv ? pdl::load(p + i) : make_uint2(0u, 0u);
      }
    };
    if (a.gate != nullptr) fetch(a.gate + static_cast<long long>(rc / a.period) * a.nv, gate);
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int i = tr + k * TPR;
      y[k][0] = y[k][1] = make_float2(0.0f, 0.0f);
      if (active && i < a.nv) staged22<YB>(staged, i, y[k]);
    }
    float r1 = 1.0f;
    if (a.g_post != nullptr) {
      fetch(a.g_post, gain);
      double ss = sum_squares(y);
      ss = bn_reduce<TPR, THREADS, double>(ss, s_y, rib, false);
      r1 = bn_rstd(ss, d, eps);
      const float2 r1v = splat2(r1);
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        y[k][0] = mul2(mul2(y[k][0], r1v), unpack2(gain[k].x));
        y[k][1] = mul2(mul2(y[k][1], r1v), unpack2(gain[k].y));
      }
    }
    if (a.gate != nullptr) {
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        y[k][0] = mul2(unpack2(gate[k].x), y[k][0]);
        y[k][1] = mul2(unpack2(gate[k].y), y[k][1]);
      }
    }
    fetch(a.g_pre, gain);
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int i = tr + k * TPR;
      if (active && i < a.nv) {
        float2 h[2];
        staged22<!HF>(staged + y_bytes, i, h);
        // y is h' from here on
#pragma unroll
        for (int j = 0; j < 2; ++j)
          y[k][j] = make_float2(__fadd_rn(__fmul_rn(a.res_scale, h[j].x), y[k][j].x),
                                __fadd_rn(__fmul_rn(a.res_scale, h[j].y), y[k][j].y));
        if constexpr (HF) {
          static_cast<float4*>(a.H_out)[at + i] = make_float4(y[k][0].x, y[k][0].y, y[k][1].x, y[k][1].y);
        } else {
          const uint2 w = make_uint2(pack2(y[k][0]), pack2(y[k][1]));
          static_cast<uint2*>(a.H_out)[at + i] = w;
          y[k][0] = unpack2(w.x);
          y[k][1] = unpack2(w.y);
        }
      } else {
        y[k][0] = y[k][1] = make_float2(0.0f, 0.0f);
      }
    }
    double ss = sum_squares(y);
    ss = bn_reduce<TPR, THREADS, double>(ss, s_h, rib, false);
    // every thread of the group has its columns in registers
    if (tr == 0 && row + a.depth * stride < a.T) request(row + a.depth * stride, slot);
    const float r2 = bn_rstd(ss, d, eps);
    const float2 r2v = splat2(r2);
    uint32_t mx = 0u;
    uint2 xn[VPT];
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int i = tr + k * TPR;
      xn[k] = make_uint2(pack2(mul2(mul2(y[k][0], r2v), unpack2(gain[k].x))),
                         pack2(mul2(mul2(y[k][1], r2v), unpack2(gain[k].y))));
      if (i < a.nv) {
        mx = __vmaxu2(mx, __vmaxu2(xn[k].x & 0x7FFF7FFFu, xn[k].y & 0x7FFF7FFFu));
        if (active && a.Xn != nullptr) a.Xn[at + i] = xn[k];
      }
    }
    mx = max(mx & 0xFFFFu, mx >> 16);
    mx = bn_reduce<TPR, THREADS, uint32_t>(mx, s_max, rib, true);
    // magnitudes order like their bits with infinity and NaN on top, so amax is one of them
    // where the row holds one; its codes are then 0 and every product of the row is NaN
    float am = __uint_as_float(mx << 16);
    if (am < 1e-5f) am = 1e-5f;
    if (active && tr == 0) {
      if (a.amax != nullptr) a.amax[row] = am;
      if (a.rstd != nullptr) {
        a.rstd[row] = r1;
        a.rstd[a.T + row] = r2;
      }
    }
    if (active && a.Xq != nullptr) {
      const bool finite = mx < 0x7F80u;
      const float sc = __fdiv_rn(127.0f, am);
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        const int i = tr + k * TPR;
        if (i >= a.nv) continue;
        const float2 x0 = unpack2(xn[k].x), x1 = unpack2(xn[k].y);
        const uint32_t q0 = code(x0.x, sc), q1 = code(x0.y, sc), q2 = code(x1.x, sc), q3 = code(x1.y, sc);
        const uint32_t w = __byte_perm(__byte_perm(q0, q1, 0x0040u), __byte_perm(q2, q3, 0x0040u), 0x5410u);
        a.Xq[at + i] = finite ? w : 0u;
      }
    }
  }
}

constexpr int kBnMaxDepth = 4;

template <int TPR, int VPT, bool YB, bool HF>
cudaError_t run(BlockNormArgs a, cudaStream_t stream, int num_sms) {
  constexpr int THREADS = bn_threads(TPR), RPB = THREADS / TPR, blocks_per_sm = bn_blocks(TPR, VPT);
  long long blocks = (static_cast<long long>(a.T) + RPB - 1) / RPB;
  const long long cap = static_cast<long long>(num_sms) * blocks_per_sm;
  if (blocks > cap) blocks = cap;
  // as many rows ahead as the block's share of shared memory holds, and no more than it has rows
  const int slot = a.nv * ((YB ? 8 : 16) + (HF ? 16 : 8)) * RPB;
  const int budget = 220 * 1024 / blocks_per_sm - 1024;
  const long long rows = (static_cast<long long>(a.T) + blocks * RPB - 1) / (blocks * RPB);
  a.depth = budget / slot < kBnMaxDepth ? budget / slot : kBnMaxDepth;
  if (a.depth > rows) a.depth = static_cast<int>(rows);
  if (a.depth < 1) a.depth = 1;
  const int smem = a.depth * slot + RPB * a.depth * 8;
  auto kern = block_norm_kernel<TPR, VPT, YB, HF>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 220 * 1024);
  if (e != cudaSuccess) return e;
  return pdl::launch(kern, static_cast<int>(blocks), THREADS, smem, 1, stream, a);
}

// Threads per row and vectors per thread.  Few rows want many threads per row (latency), many rows few
// (what every thread does once per row, the sums and two square roots, is shared by more columns), and as
// many vectors as the width fills: a vector past the row's end costs what a full one costs.
// Measured, this choice against the other side of each rule, y fp32 and h bf16 unless said:
//   many rows, vectors by the width against always 8 (4 with an fp32 stream), 67 MB of y each: 528 columns
//     79.6 us against 110, 1040 79.3 against 108, 1280 66 against 86, 2064 82 against 112, 5120 68 against 81;
//   an fp32 stream: 5 vectors of the narrower shape against 3 of the wider: 528 columns 79.3 us against
//     98.5, 1280 72.5 against 83.6; beyond 5 they leave the ring too shallow: 2048 columns, 16000 rows
//     79.3 with 64 threads of 8 against 72.5 with 128 of 4;
//   8 or 16 threads against 32: 128 columns, 8192 rows 7.1 us, 32768 rows 14.5 against 21.6, 131072 rows
//     37 against 78; 272 columns, 15420 rows 16.8 against 15.8, 61680 rows 41.8 against 50.6;
//     512 columns, 65536 rows 66.5 with 16 of 8 against 64.0 with 32 of 4;
//   896 columns: 1 row 2.4 us with 256 threads, 2.6 with 128; 1000 rows 4.4 with 128, 5.9 with 4 vectors
//     each; 16000 rows 31.5 with 32 of 8 (7 fill it), 35.1 with 64 of 4;
//   2048 columns: 300 rows 3.7 us with 256 threads, 4.5 with 64 of 8; 16000 rows 60.3 with 64 of 8,
//     68.5 with 128 of 4;
//   4096 columns: 300 rows 4.7 us with 256 of 4, 5.6 with 128 of 8; 16000 rows 126 against 117;
//   8192 columns: 300 rows 8.1 us with 256 of 8, 9.9 with 512 of 4; 1 row 4.2 against 4.0.

// 5 to 8 vectors for rows of more than 4 TPR vectors.
template <int TPR, bool YB, bool HF>
cudaError_t run_wide(const BlockNormArgs& a, cudaStream_t stream, int num_sms) {
  if (a.nv <= 5 * TPR) return run<TPR, 5, YB, HF>(a, stream, num_sms);
  if (a.nv <= 6 * TPR) return run<TPR, 6, YB, HF>(a, stream, num_sms);
  if (a.nv <= 7 * TPR) return run<TPR, 7, YB, HF>(a, stream, num_sms);
  return run<TPR, 8, YB, HF>(a, stream, num_sms);
}

// 3 or 4 vectors for rows of more than 2 TPR.
template <int TPR, bool YB, bool HF>
cudaError_t run_narrow(const BlockNormArgs& a, cudaStream_t stream, int num_sms) {
  return a.nv <= 3 * TPR ? run<TPR, 3, YB, HF>(a, stream, num_sms) : run<TPR, 4, YB, HF>(a, stream, num_sms);
}

// Many rows of more than 4 TPR and at most 8 TPR vectors.
template <int TPR, bool YB, bool HF>
cudaError_t run_many(const BlockNormArgs& a, cudaStream_t stream, int num_sms) {
  if constexpr (HF) {
    if (a.nv > 5 * TPR) return run_narrow<2 * TPR, YB, HF>(a, stream, num_sms);
    return run<TPR, 5, YB, HF>(a, stream, num_sms);
  } else {
    return run_wide<TPR, YB, HF>(a, stream, num_sms);
  }
}

template <bool YB, bool HF>
cudaError_t dispatch(const BlockNormArgs& a, cudaStream_t stream, int num_sms) {
  const bool many = a.T > 4 * num_sms, very_many = a.T > 160 * num_sms;
  if (a.nv <= 64) {
    if (!very_many) return run<32, 2, YB, HF>(a, stream, num_sms);
    if (a.nv <= 32) return run<8, 4, YB, HF>(a, stream, num_sms);
    return run_many<8, YB, HF>(a, stream, num_sms);
  }
  if (a.nv <= 128) {
    if (!many) return run<64, 2, YB, HF>(a, stream, num_sms);
    if (very_many && a.nv <= 112) return run_many<16, YB, HF>(a, stream, num_sms);
    return run_narrow<32, YB, HF>(a, stream, num_sms);
  }
  if (a.nv <= 256 && a.T > num_sms)
    return many ? run_many<32, YB, HF>(a, stream, num_sms) : run<128, 2, YB, HF>(a, stream, num_sms);
  if (a.nv <= 512)
    return many ? run_many<64, YB, HF>(a, stream, num_sms) : run<256, 2, YB, HF>(a, stream, num_sms);
  if (a.nv <= 1024)
    return many ? run_many<128, YB, HF>(a, stream, num_sms) : run_narrow<256, YB, HF>(a, stream, num_sms);
  if (a.nv <= 2048)
    return a.T > num_sms ? run_wide<256, YB, HF>(a, stream, num_sms) : run<512, 4, YB, HF>(a, stream, num_sms);
  return run_wide<512, YB, HF>(a, stream, num_sms);
}

}  // namespace

cudaError_t launch_block_norm(const BlockNormDev& p, cudaStream_t stream, int num_sms, uint32_t* err) {
  if (p.T == 0) return cudaSuccess;
  BlockNormArgs a{};
  a.Y = p.Y;
  a.H = p.H;
  a.g_post = static_cast<const uint2*>(p.g_post);
  a.gate = static_cast<const uint2*>(p.gate);
  a.g_pre = static_cast<const uint2*>(p.g_pre);
  a.H_out = p.H_out;
  a.Xn = static_cast<uint2*>(p.Xn);
  a.Xq = reinterpret_cast<uint32_t*>(p.Xq);
  a.amax = p.amax;
  a.rstd = p.rstd;
  a.res_scale = p.res_scale;
  a.eps = p.eps;
  a.period = p.gate_period;
  a.T = p.T;
  a.nv = p.d / 4;
  a.err = err;
  if (p.y_bf16) return p.h_f32 ? dispatch<true, true>(a, stream, num_sms) : dispatch<true, false>(a, stream, num_sms);
  return p.h_f32 ? dispatch<false, true>(a, stream, num_sms) : dispatch<false, false>(a, stream, num_sms);
}

}  // namespace sbl
