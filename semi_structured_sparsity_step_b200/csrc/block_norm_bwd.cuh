// block_norm_bwd.cuh -- the kernel of the block norm's backward pass and its launch, for one of four
// modes (branch norm or not, gate or not), each instantiated in a file of its own.  block_norm_bwd.cu
// has the mathematics and joins the modes.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <algorithm>
#include <atomic>
#include <cstdint>

#include "block_norm.cuh"
#include "sbl_device.cuh"
#include "sbl_internal.h"

namespace sbl {

constexpr int kBbMaxSms = 160;  // sizes the workspace
constexpr int kBbWaves = 4;     // segments per row lane at most

struct BwdArgs {
  const float* dXn[3];
  const void* dH_in;     // may be NULL (zero)
  const void* Y;         // not read without a branch norm and dgate
  const void* H;         // h'
  const uint2* g_post;   // may be NULL
  const uint2* gate;     // may be NULL
  const uint2* g_pre;
  const float* rstd;     // [2, T]
  uint2* dY;
  void* dH;              // may be NULL
  float4* part_pre;      // [blocks, d]
  float4* part_post;     // [blocks, d]
  float4* gate_out;      // [segments, d]: dgate itself when a group is one segment, else partial rows
  int gate_accumulate;   // gate_out is dgate and is added to
  int readers;
  float res_scale;
  int T, nv, vecs_per_cta;
  int period, seg_rows, segs_per_group, segs;  // tokens per gate row, rows per segment
  int depth, slot_bytes; // rows of the ring, bytes of a block's slice of a staged row (at most)
  int col_bytes;         // staged bytes per column
  uint32_t* err;
};

struct GradOut {
  float4* ws;
  float* dgate;
  bool pre, post;
  int accumulate;
};

// The four modes; `blocks` receives how many partial rows each gain's gradient has.
cudaError_t block_norm_bwd_plain(BwdArgs& a, const GradOut& g, bool y_bf16, bool h_f32, int& blocks,
                                 cudaStream_t stream, int num_sms);
cudaError_t block_norm_bwd_gate(BwdArgs& a, const GradOut& g, bool y_bf16, bool h_f32, int& blocks,
                                cudaStream_t stream, int num_sms);
cudaError_t block_norm_bwd_post(BwdArgs& a, const GradOut& g, bool y_bf16, bool h_f32, int& blocks,
                                cudaStream_t stream, int num_sms);
cudaError_t block_norm_bwd_post_gate(BwdArgs& a, const GradOut& g, bool y_bf16, bool h_f32, int& blocks,
                                     cudaStream_t stream, int num_sms);

// Row lanes of the whole grid at most, over the shapes that a width can take (12 columns per thread and
// the fewest threads).
inline int max_units(int d, int sms) {
  if (d <= 3 * 128) return 16 * sms;
  if (d <= 3 * 256) return 8 * sms;
  if (d <= 3 * 512) return 4 * sms;
  if (d <= 4096) return 2 * sms;
  return sms;
}

namespace {

// Blocks of 256 threads, two per SM, or of the 512 that share one row, one per SM.
constexpr int bb_threads(int tpr) { return tpr < 256 ? 256 : tpr; }
constexpr int bb_blocks_per_sm(int tpr) { return tpr > 256 ? 1 : 2; }
constexpr int bb_ring_bytes(int tpr) { return tpr > 256 ? 224 * 1024 : 108 * 1024; }

template <int TPR, int VPT, int CS, bool YB, bool HF, bool POST, bool GATE>
__global__ void __launch_bounds__(bb_threads(TPR), bb_blocks_per_sm(TPR)) block_norm_bwd_kernel(const BwdArgs a) {
  constexpr int THREADS = bb_threads(TPR);
  constexpr int RPB = THREADS / TPR;   // row lanes
  constexpr int WPR = TPR / 32;        // warps of a row lane
  constexpr int SLOTS = CS * WPR;      // warps that share a row
  __shared__ float s_sum[2][(CS > 1 ? SLOTS : THREADS / 32) * 4];  // three sums per warp
  __shared__ int s_abort;
  __shared__ float4 s_zero;  // four columns of a gradient that is not given
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rib = threadIdx.x / TPR;
  const int tr = threadIdx.x % TPR;
  const int rank = CS > 1 ? static_cast<int>(pair::cluster_rank()) : 0;
  const int unit = static_cast<int>(blockIdx.x) / CS * RPB + rib;  // row lane of the grid
  const int units = static_cast<int>(gridDim.x) / CS * RPB;
  const int first_vec = rank * a.vecs_per_cta;
  const int my_vecs = min(a.vecs_per_cta, a.nv - first_vec);  // this block's slice of a row
  const float inv_d = 1.0f / (4.0f * static_cast<float>(a.nv));
  // one staged row: y (if needed), h', dH (if given), the readers' gradients, the gate row (if given)
  const uint32_t b16 = static_cast<uint32_t>(my_vecs) * 8u, b32 = 2u * b16;
  const bool with_y = POST || a.gate_out != nullptr;
  const uint32_t y_bytes = !with_y ? 0u : YB ? b16 : b32, h_bytes = HF ? b32 : b16;
  const uint32_t off_dh = y_bytes + h_bytes;
  const uint32_t off_dx = off_dh + (a.dH_in != nullptr ? h_bytes : 0u);
  const uint32_t off_gate = off_dx + static_cast<uint32_t>(a.readers) * b32;
  const uint32_t row_bytes = off_gate + (GATE ? b16 : 0u);
  extern __shared__ __align__(128) uint8_t ring[];
  uint8_t* slots = ring + static_cast<size_t>(rib) * a.depth * a.slot_bytes;
  uint64_t* bars =
      reinterpret_cast<uint64_t*>(ring + static_cast<size_t>(RPB) * a.depth * a.slot_bytes) + rib * a.depth;
  if (tr == 0) {
    for (int i = 0; i < a.depth; ++i) mbar_init(&bars[i], 1);
    s_abort = 0;
    s_zero = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    fence_mbar_init();
  }
  const int dh_mask = a.dH_in != nullptr ? -1 : 0;
  auto request = [&](int row, int slot) {
    uint8_t* dst = slots + static_cast<size_t>(slot) * a.slot_bytes;
    uint64_t* bar = &bars[slot];
    const long long at = (static_cast<long long>(row) * a.nv + first_vec) * 4;
    mbar_arrive_expect_tx(bar, row_bytes);
    if (with_y) bulk_load(dst, static_cast<const uint8_t*>(a.Y) + at * (YB ? 2 : 4), y_bytes, bar);
    bulk_load(dst + y_bytes, static_cast<const uint8_t*>(a.H) + at * (HF ? 4 : 2), h_bytes, bar);
    if (a.dH_in != nullptr)
      bulk_load(dst + off_dh, static_cast<const uint8_t*>(a.dH_in) + at * (HF ? 4 : 2), h_bytes, bar);
    for (int q = 0; q < a.readers; ++q) bulk_load(dst + off_dx + q * b32, a.dXn[q] + at, b32, bar);
    if constexpr (GATE) {
      const long long gat = (static_cast<long long>(row / a.period) * a.nv + first_vec) * 4;
      bulk_load(dst + off_gate, reinterpret_cast<const uint8_t*>(a.gate) + gat * 2, b16, bar);
    }
  };
  __syncthreads();
  if constexpr (CS > 1) pair::cluster_sync();  // every block of the cluster is there
  pdl::wait();

  // Every row lane walks its segments, seg_rows steps each (steps past a segment's rows are
  // inactive), so all blocks of a cluster take the same number of steps and barriers.
  struct Walk {
    int seg, step, row, rows;  // rows: how many of the segment's steps are active
  };
  auto enter = [&](Walk& w) {
    w.step = 0;
    w.row = w.rows = 0;
    if (w.seg < a.segs) {
      const int group = w.seg / a.segs_per_group;
      const long long in_group = static_cast<long long>(w.seg - group * a.segs_per_group) * a.seg_rows;
      const long long first = static_cast<long long>(group) * a.period + in_group;
      const long long left = min(static_cast<long long>(a.period) - in_group, static_cast<long long>(a.T) - first);
      w.row = static_cast<int>(min(first, static_cast<long long>(a.T)));
      w.rows = static_cast<int>(max(0ll, min(left, static_cast<long long>(a.seg_rows))));
    }
  };
  // The requests run ahead of the arithmetic through the same sequence of active rows.
  Walk ahead{unit, 0, 0, 0}, w{unit, 0, 0, 0};
  enter(w);
  RingPos fill, pos;
  auto request_next = [&]() {
    while (ahead.step >= ahead.rows) {
      if (ahead.seg >= a.segs) return;
      ahead.seg += units;
      enter(ahead);
    }
    request(ahead.row + ahead.step, fill.slot);
    ++ahead.step;
    fill.next(a.depth);
  };
  if (tr == 0) {
    enter(ahead);
    for (int i = 0; i < a.depth; ++i) request_next();
  }

  uint2 gpre[VPT], gpost[VPT];
  float2 acc_pre[VPT][2], acc_post[POST ? VPT : 1][2], acc_gate[GATE ? VPT : 1][2];
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const int i = tr + k * TPR;
    gpre[k] = gpost[k] = make_uint2(0x3F803F80u, 0x3F803F80u);  // 1.0
    if (i < my_vecs) {
      gpre[k] = a.g_pre[first_vec + i];
      if constexpr (POST) gpost[k] = a.g_post[first_vec + i];
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      acc_pre[k][j] = make_float2(0.0f, 0.0f);
      if constexpr (POST) acc_post[k][j] = make_float2(0.0f, 0.0f);
      if constexpr (GATE) acc_gate[k][j] = make_float2(0.0f, 0.0f);
    }
  }
  const int rounds = (a.segs + units - 1) / units;
  int buf = 0;
  for (int rd = 0; rd < rounds; ++rd) {
    for (int step = 0; step < a.seg_rows; ++step) {
      const bool active = step < w.rows;
      const int row = w.row + step;
      float r1 = 1.0f, r2 = 0.0f;
      if (active) {
        if constexpr (POST) r1 = a.rstd[row];
        r2 = a.rstd[static_cast<long long>(a.T) + row];
      }
      const uint8_t* staged = slots + static_cast<size_t>(pos.slot) * a.slot_bytes;
      const uint8_t* s_dh = a.dH_in != nullptr ? staged + off_dh : reinterpret_cast<const uint8_t*>(&s_zero);
      const uint2* s_gate = reinterpret_cast<const uint2*>(staged + off_gate);
      float2 t[VPT][2];
      float2 s2v = make_float2(0.0f, 0.0f), sav = s2v, sbv = s2v;
      if (active) {
        mbar_wait(&bars[pos.slot], pos.parity, &s_abort, a.err);
        pos.next(a.depth);
        const float2 r1v = splat2(r1), r2v = splat2(r2);
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
          const int i = tr + k * TPR;
          if (i >= my_vecs) continue;
          float2 h[2], y[2], dh[2], more[2];
          staged22<false>(staged + off_dx, i, t[k]);
          if (a.readers > 1) {
            staged22<false>(staged + off_dx + b32, i, more);
            t[k][0] = add2(t[k][0], more[0]);
            t[k][1] = add2(t[k][1], more[1]);
          }
          if (a.readers > 2) {
            staged22<false>(staged + off_dx + 2 * b32, i, more);
            t[k][0] = add2(t[k][0], more[0]);
            t[k][1] = add2(t[k][1], more[1]);
          }
          staged22<!HF>(staged + y_bytes, i, h);
          uint2 gt = make_uint2(0u, 0u);
          if constexpr (POST) {
            staged22<YB>(staged, i, y);
            staged22<!HF>(s_dh, i & dh_mask, dh);
            if constexpr (GATE) gt = s_gate[i];
          }
          const uint32_t gw[2] = {gpre[k].x, gpre[k].y}, pw[2] = {gpost[k].x, gpost[k].y}, tw[2] = {gt.x, gt.y};
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float2 xh = mul2(h[j], r2v);
            acc_pre[k][j] = fma2(t[k][j], xh, acc_pre[k][j]);
            t[k][j] = mul2(t[k][j], unpack2(gw[j]));
            s2v = fma2(t[k][j], xh, s2v);
            if constexpr (POST) {
              float2 wt = mul2(unpack2(pw[j]), mul2(y[j], r1v));
              if constexpr (GATE) wt = mul2(unpack2(tw[j]), wt);
              sav = fma2(wt, fma2(r2v, t[k][j], dh[j]), sav);
              sbv = fma2(wt, xh, sbv);
            }
          }
        }
      }

      // The three sums of the warp meet in lanes 0, 8 and 16 (lane >> 3 is the sum, 3 is none): halving
      // what a lane carries at each step takes 6 shuffles where three full sums take 15.
      float s2, sa = 0.0f, sb = 0.0f, part;
      if constexpr (POST) {
        const float v0 = s2v.x + s2v.y, v1 = sav.x + sav.y, v2 = sbv.x + sbv.y;
        const bool up = (lane & 16) != 0, up2 = (lane & 8) != 0;
        float k0 = (up ? v2 : v0) + __shfl_xor_sync(0xFFFFFFFFu, up ? v0 : v2, 16);
        float k1 = (up ? 0.0f : v1) + __shfl_xor_sync(0xFFFFFFFFu, up ? v1 : 0.0f, 16);
        part = (up2 ? k1 : k0) + __shfl_xor_sync(0xFFFFFFFFu, up2 ? k0 : k1, 8);
      } else {
        part = s2v.x + s2v.y;
        part += __shfl_xor_sync(0xFFFFFFFFu, part, 16);
        part += __shfl_xor_sync(0xFFFFFFFFu, part, 8);
      }
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) part += __shfl_xor_sync(0xFFFFFFFFu, part, o);
      if constexpr (SLOTS > 1) {
        const bool holds = (lane & 7) == 0;
        if constexpr (CS > 1) {
          if (holds) {
            const uint32_t own = smem_u32(&s_sum[buf][(rank * WPR + warp) * 4 + (lane >> 3)]);
#pragma unroll
            for (uint32_t p = 0; p < CS; ++p)
              asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(pair::map_to(own, p)), "f"(part) : "memory");
          }
          __syncwarp();
          pair::cluster_sync();
        } else {
          if (holds) s_sum[buf][warp * 4 + (lane >> 3)] = part;
          lane_sync<TPR, THREADS>(rib);
        }
        // lane 8 c + w adds up sum c of warps w, w + 8, ...
        const float* sums = s_sum[buf] + (CS > 1 ? 0 : rib * WPR * 4) + (lane >> 3);
        part = 0.0f;
#pragma unroll
        for (int w = 0; w < SLOTS; w += 8)
          if (SLOTS >= 8 || (lane & 7) < SLOTS) part += sums[(w + (lane & 7)) * 4];
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) part += __shfl_xor_sync(0xFFFFFFFFu, part, o);
      } else {
        __syncwarp();
      }
      s2 = __shfl_sync(0xFFFFFFFFu, part, 0);
      if constexpr (POST) {
        sa = __shfl_sync(0xFFFFFFFFu, part, 8);
        sb = __shfl_sync(0xFFFFFFFFu, part, 16);
      }
      buf ^= 1;  // two buffers: a warp can be at most one barrier ahead of another's reads
      if (active) {
        const float c2 = s2 * inv_d;
        const float c1 = fmaf(-r2 * c2, sb, sa) * inv_d;
        const float2 r1v = splat2(r1), r2v = splat2(r2), k2 = splat2(-r2 * r2 * c2), k1 = splat2(-r1 * c1),
                     scale = splat2(a.res_scale);
        const long long at = static_cast<long long>(row) * a.nv + first_vec;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
          const int i = tr + k * TPR;
          if (i >= my_vecs) continue;
          float2 h[2], y[2], dh[2], dy[2];
          staged22<!HF>(staged + y_bytes, i, h);
          staged22<!HF>(s_dh, i & dh_mask, dh);
          if constexpr (POST || GATE) staged22<YB>(staged, i, y);
          uint2 gt = make_uint2(0u, 0u);
          if constexpr (GATE) gt = s_gate[i];
          const uint32_t pw[2] = {gpost[k].x, gpost[k].y}, tw[2] = {gt.x, gt.y};
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float2 d = fma2(h[j], k2, fma2(r2v, t[k][j], dh[j]));
            dh[j] = mul2(scale, d);
            float2 du = d;
            if constexpr (GATE) du = mul2(unpack2(tw[j]), d);
            if constexpr (POST) {
              const float2 gp = unpack2(pw[j]), yh = mul2(y[j], r1v);
              if constexpr (GATE) acc_gate[k][j] = fma2(d, mul2(yh, gp), acc_gate[k][j]);
              acc_post[k][j] = fma2(du, yh, acc_post[k][j]);
              dy[j] = fma2(yh, k1, mul2(r1v, mul2(du, gp)));
            } else {
              if constexpr (GATE) acc_gate[k][j] = fma2(d, y[j], acc_gate[k][j]);
              dy[j] = du;
            }
          }
          a.dY[at + i] = make_uint2(pack2(dy[0]), pack2(dy[1]));
          if (a.dH != nullptr) {
            if constexpr (HF)
              static_cast<float4*>(a.dH)[at + i] = make_float4(dh[0].x, dh[0].y, dh[1].x, dh[1].y);
            else
              static_cast<uint2*>(a.dH)[at + i] = make_uint2(pack2(dh[0]), pack2(dh[1]));
          }
        }
        // the slot is free once every thread of the lane is past its second read (the values went into
        // what it has stored or added up)
        lane_sync<TPR, THREADS>(rib);
        if (tr == 0) request_next();
      }
    }
    if constexpr (GATE) {
      const bool there = a.gate_out != nullptr && w.seg < a.segs;
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        const int i = tr + k * TPR;
        if (there && i < my_vecs) {
          float4* out = a.gate_out + static_cast<long long>(w.seg) * a.nv + first_vec + i;
          float4 v = make_float4(acc_gate[k][0].x, acc_gate[k][0].y, acc_gate[k][1].x, acc_gate[k][1].y);
          if (a.gate_accumulate) {
            const float4 o = *out;
            v = make_float4(o.x + v.x, o.y + v.y, o.z + v.z, o.w + v.w);
          }
          *out = v;
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) acc_gate[k][j] = make_float2(0.0f, 0.0f);
      }
    }
    w.seg += units;
    enter(w);
  }

  // the block's row lanes meet in shared memory (the ring's, every staged row is consumed): one
  // partial row per block
  float4* s_col = reinterpret_cast<float4*>(ring);
  auto leave = [&](const auto& acc, float4* part) {
    __syncthreads();
#pragma unroll
    for (int k = 0; k < VPT; ++k)
      s_col[(rib * VPT + k) * TPR + tr] = make_float4(acc[k][0].x, acc[k][0].y, acc[k][1].x, acc[k][1].y);
    __syncthreads();
    for (int c = threadIdx.x; c < my_vecs; c += THREADS) {
      float4 s = s_col[c];
#pragma unroll
      for (int r = 1; r < RPB; ++r) {
        const float4 v = s_col[r * VPT * TPR + c];
        s = make_float4(s.x + v.x, s.y + v.y, s.z + v.z, s.w + v.w);
      }
      part[static_cast<long long>(blockIdx.x / CS) * a.nv + first_vec + c] = s;
    }
  };
  if (a.part_pre != nullptr) leave(acc_pre, a.part_pre);
  if constexpr (POST) {
    if (a.part_post != nullptr) leave(acc_post, a.part_post);
  }
}

constexpr int kBbMaxDepth = 4;

// How many clusters of this kernel are resident at once: fewer than the SMs alone would hold, as a
// cluster stays within one group of SMs.  Asked once per device.
template <typename Kern>
int resident_clusters(Kern kern, int threads, int cs, int smem, int num_sms, std::atomic<int> (&cached)[64]) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return num_sms / cs;
  int n = cached[dev].load();
  if (n == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(cs));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(cs);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n < 1) n = num_sms / cs;
    n = std::min(n, num_sms / cs);
    cached[dev].store(n);
  }
  return n;
}

// Cuts each group of tokens that share a gate row into segs_per_group segments: the choice with the
// fewest steps on the busiest row lane, a segment's end counted as half a step.
void cut_segments(BwdArgs& a, int units) {
  const int groups = (a.T + a.period - 1) / a.period;
  double best = 1e30;
  for (int w = 0; w <= kBbWaves; ++w) {
    long long s = w == 0 ? 1 : static_cast<long long>(w) * units / groups;
    s = std::max(1ll, std::min(s, static_cast<long long>(a.period)));
    const int rows = static_cast<int>((a.period + s - 1) / s);
    const int per_group = (a.period + rows - 1) / rows;
    const long long segs = static_cast<long long>(groups) * per_group;
    const double cost = static_cast<double>((segs + units - 1) / units) * (rows + (a.gate != nullptr ? 0.5 : 0.0));
    if (cost < best) {
      best = cost;
      a.seg_rows = rows;
      a.segs_per_group = per_group;
      a.segs = static_cast<int>(segs);
    }
  }
}

template <int TPR, int VPT, int CS, bool YB, bool HF, bool POST, bool GATE>
cudaError_t run_typed(BwdArgs& a, const GradOut& g, int& blocks, cudaStream_t stream, int num_sms) {
  constexpr int THREADS = bb_threads(TPR), RPB = THREADS / TPR, RING = bb_ring_bytes(TPR);
  auto kern = block_norm_bwd_kernel<TPR, VPT, CS, YB, HF, POST, GATE>;
  const int smem_max = RING + 128;  // the barriers of two rows of 8 lanes behind the ring
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_max);
  if (e != cudaSuccess) return e;
  int clusters = bb_blocks_per_sm(TPR) * num_sms / CS;
  if constexpr (CS > 1) {
    static std::atomic<int> cached[64];
    clusters = resident_clusters(kern, THREADS, CS, smem_max, num_sms, cached);
  }
  const int units_max = clusters * RPB;
  cut_segments(a, units_max);
  const int units = a.segs < units_max ? a.segs : units_max;
  blocks = (units + RPB - 1) / RPB;
  // a multiple of 16 columns, so that every block's slice of a row starts and ends on 16 bytes
  a.vecs_per_cta = CS > 1 ? (a.nv / 4 + CS - 1) / CS * 4 : a.nv;
  a.slot_bytes = a.vecs_per_cta * a.col_bytes * 4;
  a.depth = std::max(1, std::min(kBbMaxDepth, (RING + 128) / (RPB * (a.slot_bytes + 8))));
  const int smem = std::max(RPB * a.depth * (a.slot_bytes + 8), THREADS * VPT * 16 /* the column sums at the end */);
  // where the partial rows go
  const size_t rows = static_cast<size_t>(max_units(a.nv * 4, kBbMaxSms));
  if (g.pre) a.part_pre = g.ws;
  if (g.post) a.part_post = g.ws + rows * a.nv;
  if (g.dgate != nullptr) {
    a.gate_out = a.segs_per_group > 1 ? g.ws + 2 * rows * a.nv : reinterpret_cast<float4*>(g.dgate);
    a.gate_accumulate = a.segs_per_group > 1 ? 0 : g.accumulate;
  }
  return pdl::launch(kern, blocks * CS, THREADS, smem, CS, stream, a);
}

template <int TPR, int VPT, int CS, bool POST, bool GATE>
cudaError_t run(BwdArgs& a, const GradOut& g, bool yb, bool hf, int& blocks, cudaStream_t stream, int num_sms) {
  if constexpr (POST || GATE) {  // y is read
    if (yb)
      return hf ? run_typed<TPR, VPT, CS, true, true, POST, GATE>(a, g, blocks, stream, num_sms)
                : run_typed<TPR, VPT, CS, true, false, POST, GATE>(a, g, blocks, stream, num_sms);
  }
  return hf ? run_typed<TPR, VPT, CS, false, true, POST, GATE>(a, g, blocks, stream, num_sms)
            : run_typed<TPR, VPT, CS, false, false, POST, GATE>(a, g, blocks, stream, num_sms);
}

// Whether two rows can be staged for every row lane of TPR threads.
inline bool stages_two(const BwdArgs& a, int tpr) {
  return 2 * (bb_threads(tpr) / tpr) * a.nv * 4 * a.col_bytes <= bb_ring_bytes(tpr);
}

// Threads per row and vectors per thread: columns that a row does not fill cost what full ones cost, so
// 12 columns per thread where they hold a row that 8 do not, and 16 beyond 2048 columns, as long as two
// rows can be staged.  Measured against 8 (16 beyond 2048) alone, 67 MB of y: bf16, one reader: 272 columns
// 106 us against 150, 528 107 against 154, 1040 112 against 139, 5120 85 against 94; y fp32, a gate row per
// token, two readers: 528 columns 167 against 235, 2064 145 against 223, 5120 133 against 240 (a cluster).
// With a row per SM or less 12 columns lose: 126 x 1040 6.0 us against 5.5.  16 columns below 2049: 16384 x
// 2048, bf16, one reader 115 us against 98.  Clusters of blocks of 256 threads, two per SM, in place of
// 512: 8192 columns 240 us against 172.
template <bool POST, bool GATE>
cudaError_t run_mode(BwdArgs& a, const GradOut& g, bool yb, bool hf, int& blocks, cudaStream_t stream, int num_sms) {
  const int nv = a.nv;
  const auto by_12 = [&](int tpr) { return nv <= 3 * tpr && a.T > num_sms && stages_two(a, tpr); };
  if (nv <= 64) return run<32, 2, 1, POST, GATE>(a, g, yb, hf, blocks, stream, num_sms);
  if (by_12(32)) return run<32, 3, 1, POST, GATE>(a, g, yb, hf, blocks, stream, num_sms);
  if (nv <= 128) return run<64, 2, 1, POST, GATE>(a, g, yb, hf, blocks, stream, num_sms);
  if (by_12(64)) return run<64, 3, 1, POST, GATE>(a, g, yb, hf, blocks, stream, num_sms);
  if (nv <= 256) return run<128, 2, 1, POST, GATE>(a, g, yb, hf, blocks, stream, num_sms);
  if (by_12(128)) return run<128, 3, 1, POST, GATE>(a, g, yb, hf, blocks, stream, num_sms);
  if (nv <= 512) return run<256, 2, 1, POST, GATE>(a, g, yb, hf, blocks, stream, num_sms);
  if (nv <= 768 && stages_two(a, 256)) return run<256, 3, 1, POST, GATE>(a, g, yb, hf, blocks, stream, num_sms);
  if (nv <= 1024)
    return stages_two(a, 256) ? run<256, 4, 1, POST, GATE>(a, g, yb, hf, blocks, stream, num_sms)
                              : run<512, 2, 1, POST, GATE>(a, g, yb, hf, blocks, stream, num_sms);
  if (nv <= 1536 && stages_two(a, 512)) return run<512, 3, 1, POST, GATE>(a, g, yb, hf, blocks, stream, num_sms);
  if (nv <= 2048)
    return stages_two(a, 512) ? run<512, 4, 1, POST, GATE>(a, g, yb, hf, blocks, stream, num_sms)
                              : run<512, 2, 2, POST, GATE>(a, g, yb, hf, blocks, stream, num_sms);
  return a.col_bytes <= 13 ? run<512, 4, 2, POST, GATE>(a, g, yb, hf, blocks, stream, num_sms)
                           : run<512, 2, 4, POST, GATE>(a, g, yb, hf, blocks, stream, num_sms);
}

}  // namespace

}  // namespace sbl
