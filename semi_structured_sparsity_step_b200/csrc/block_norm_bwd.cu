// block_norm_bwd.cu -- the backward pass of the block norm (block_norm.cu) on sm_100a.
//
// The straight-through estimator passes the quantiser by (Sparse-BitNet summary
// "Sparse-BitNet：1.58-bit 大模型天然兼容半结构化稀疏", 前置知识 (STE)), so the gradient of xn is the sum of
// the dX of the products that read it.  With the saved factors r1, r2 of a row, yh = y r1,
// xh = h' r2 and t = dxn g_pre:
//   c2 = mean(t xh),            dh' = dH + r2 (t - xh c2),      dh = s dh',
//   du = gate dh',              c1 = mean(du g_post yh),        dy = r1 (du g_post - yh c1),
//   dg_pre = sum_t dxn xh,      dg_post = sum_t du yh,          dgate = sum over its tokens of dh' yh g_post.
// c1 needs dh', which needs c2; but it is linear in c2: with w = gate g_post yh,
//   c1 = (sum w (dH + r2 t) - r2 c2 sum w xh) / d,
// so one round of three row sums serves both means, and a row costs one barrier.
//
// HBM bound: one read of each dX, dH, y and h', one write of dy and dh.  TPR threads share a row
// (a row lane), 4 VPT columns each; rows beyond 8192 columns, or too large to stage twice, go to a
// cluster of CS blocks that exchange the three sums through distributed shared memory.  A thread
// keeps its columns for all its rows, so the column sums stay in registers.  The rows to come are
// staged in a ring in shared memory by bulk copies, one ring per row lane.  A row is read from its
// slot twice, before and after the sums: only the column sums and t live in registers in between,
// which leaves room for 16 columns per thread, so the work that every thread does once per row
// (shuffles, barrier) is shared by more columns.
// Column sums leave as one partial row per block (dgate: per segment of rows with one gate row), and
// a second launch adds the partial rows in a fixed order: no atomics.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <algorithm>
#include <atomic>
#include <cstdint>

#include "block_norm.cuh"
#include "sbl_device.cuh"
#include "sbl_internal.h"

namespace sbl {
namespace {

constexpr int kBbMaxSms = 160;  // sizes the workspace
constexpr int kBbWaves = 4;     // segments per row lane at most

struct BwdArgs {
  const float* dXn[3];
  const void* dH_in;     // may be NULL (zero)
  const void* Y;
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

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
  return x;
}

// Blocks of 256 threads, two per SM, or of the 512 that share one row, one per SM.
constexpr int bb_threads(int tpr) { return tpr < 256 ? 256 : tpr; }
constexpr int bb_blocks_per_sm(int tpr) { return tpr > 256 ? 1 : 2; }
constexpr int bb_ring_bytes(int tpr) { return tpr > 256 ? 216 * 1024 : 104 * 1024; }

template <int TPR, int VPT, int CS, bool YB, bool HF>
__global__ void __launch_bounds__(bb_threads(TPR), bb_blocks_per_sm(TPR)) block_norm_bwd_kernel(const BwdArgs a) {
  constexpr int THREADS = bb_threads(TPR);
  constexpr int RPB = THREADS / TPR;   // row lanes
  constexpr int WPR = TPR / 32;        // warps of a row lane
  constexpr int SLOTS = CS * WPR;      // warps that share a row
  __shared__ float4 s_sum[2][CS > 1 ? SLOTS : THREADS / 32];
  __shared__ int s_abort;
  __shared__ float4 s_zero;  // four columns of what is not given: gradient 0, gate 1
  __shared__ uint2 s_one;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rib = threadIdx.x / TPR;
  const int tr = threadIdx.x % TPR;
  const int rank = CS > 1 ? static_cast<int>(pair::cluster_rank()) : 0;
  const int unit = static_cast<int>(blockIdx.x) / CS * RPB + rib;  // row lane of the grid
  const int units = static_cast<int>(gridDim.x) / CS * RPB;
  const int first_vec = rank * a.vecs_per_cta;
  const int my_vecs = min(a.vecs_per_cta, a.nv - first_vec);  // this block's slice of a row
  const bool post = a.g_post != nullptr;
  const float inv_d = 1.0f / (4.0f * static_cast<float>(a.nv));
  // one staged row: y, h', dH (if given), the readers' gradients, the gate row (if given)
  const uint32_t b16 = static_cast<uint32_t>(my_vecs) * 8u, b32 = 2u * b16;
  const uint32_t y_bytes = YB ? b16 : b32, h_bytes = HF ? b32 : b16;
  const uint32_t off_dh = y_bytes + h_bytes;
  const uint32_t off_dx = off_dh + (a.dH_in != nullptr ? h_bytes : 0u);
  const uint32_t off_gate = off_dx + static_cast<uint32_t>(a.readers) * b32;
  const uint32_t row_bytes = off_gate + (a.gate != nullptr ? b16 : 0u);
  extern __shared__ __align__(128) uint8_t ring[];
  uint8_t* slots = ring + static_cast<size_t>(rib) * a.depth * a.slot_bytes;
  uint64_t* bars =
      reinterpret_cast<uint64_t*>(ring + static_cast<size_t>(RPB) * a.depth * a.slot_bytes) + rib * a.depth;
  if (tr == 0) {
    for (int i = 0; i < a.depth; ++i) mbar_init(&bars[i], 1);
    s_abort = 0;
    s_zero = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    s_one = make_uint2(0x3F803F80u, 0x3F803F80u);
    fence_mbar_init();
  }
  const int dh_mask = a.dH_in != nullptr ? -1 : 0, gate_mask = a.gate != nullptr ? -1 : 0;
  auto request = [&](int row, int slot) {
    uint8_t* dst = slots + static_cast<size_t>(slot) * a.slot_bytes;
    uint64_t* bar = &bars[slot];
    const long long at = (static_cast<long long>(row) * a.nv + first_vec) * 4;
    mbar_arrive_expect_tx(bar, row_bytes);
    bulk_load(dst, static_cast<const uint8_t*>(a.Y) + at * (YB ? 2 : 4), y_bytes, bar);
    bulk_load(dst + y_bytes, static_cast<const uint8_t*>(a.H) + at * (HF ? 4 : 2), h_bytes, bar);
    if (a.dH_in != nullptr)
      bulk_load(dst + off_dh, static_cast<const uint8_t*>(a.dH_in) + at * (HF ? 4 : 2), h_bytes, bar);
    for (int q = 0; q < a.readers; ++q) bulk_load(dst + off_dx + q * b32, a.dXn[q] + at, b32, bar);
    if (a.gate != nullptr) {
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
  float2 acc_pre[VPT][2], acc_post[VPT][2], acc_gate[VPT][2];
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const int i = tr + k * TPR;
    gpre[k] = gpost[k] = make_uint2(0x3F803F80u, 0x3F803F80u);  // 1.0
    if (i < my_vecs) {
      gpre[k] = __ldg(a.g_pre + first_vec + i);
      if (post) gpost[k] = __ldg(a.g_post + first_vec + i);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) acc_pre[k][j] = acc_post[k][j] = acc_gate[k][j] = make_float2(0.0f, 0.0f);
  }
  const int rounds = (a.segs + units - 1) / units;
  int buf = 0;
  for (int rd = 0; rd < rounds; ++rd) {
    for (int step = 0; step < a.seg_rows; ++step) {
      const bool active = step < w.rows;
      const int row = w.row + step;
      float r1 = 1.0f, r2 = 0.0f;
      if (active) {
        if (post) r1 = __ldg(a.rstd + row);
        r2 = __ldg(a.rstd + a.T + row);
      }
      const uint8_t* staged = slots + static_cast<size_t>(pos.slot) * a.slot_bytes;
      const uint8_t* s_dh = a.dH_in != nullptr ? staged + off_dh : reinterpret_cast<const uint8_t*>(&s_zero);
      const uint2* s_gate = a.gate != nullptr ? reinterpret_cast<const uint2*>(staged + off_gate) : &s_one;
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
          staged22<YB>(staged, i, y);
          staged22<!HF>(s_dh, i & dh_mask, dh);
          const uint2 gt = s_gate[i & gate_mask];
          const uint32_t gw[2] = {gpre[k].x, gpre[k].y}, pw[2] = {gpost[k].x, gpost[k].y}, tw[2] = {gt.x, gt.y};
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float2 xh = mul2(h[j], r2v);
            acc_pre[k][j] = fma2(t[k][j], xh, acc_pre[k][j]);
            t[k][j] = mul2(t[k][j], unpack2(gw[j]));
            s2v = fma2(t[k][j], xh, s2v);
            const float2 wt = mul2(mul2(unpack2(tw[j]), unpack2(pw[j])), mul2(y[j], r1v));
            sav = fma2(wt, fma2(r2v, t[k][j], dh[j]), sav);
            sbv = fma2(wt, xh, sbv);
          }
        }
      }

      float s2 = warp_sum(s2v.x + s2v.y), sa = warp_sum(sav.x + sav.y), sb = warp_sum(sbv.x + sbv.y);
      if constexpr (CS > 1) {
        if (lane < CS) {
          const uint32_t dst = pair::map_to(smem_u32(&s_sum[buf][rank * WPR + warp]), static_cast<uint32_t>(lane));
          asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "f"(s2), "f"(sa), "f"(sb),
                       "f"(0.0f)
                       : "memory");
        }
        __syncwarp();
        pair::cluster_sync();
      } else if constexpr (WPR > 1) {
        if (lane == 0) s_sum[buf][warp] = make_float4(s2, sa, sb, 0.0f);
        lane_sync<TPR, THREADS>(rib);
      }
      if constexpr (SLOTS > 1) {
        // every lane takes a warp's sums (SLOTS is a power of two) and the warp adds them up
        constexpr int WIDTH = SLOTS < 32 ? SLOTS : 32;
        const float4* sums = s_sum[buf] + (CS > 1 ? 0 : rib * WPR);
        float4 v = sums[lane & (WIDTH - 1)];
        if constexpr (SLOTS > 32) {
          const float4 u = sums[lane + 32];
          v.x += u.x;
          v.y += u.y;
          v.z += u.z;
        }
#pragma unroll
        for (int o = WIDTH / 2; o > 0; o >>= 1) {
          v.x += __shfl_xor_sync(0xFFFFFFFFu, v.x, o);
          v.y += __shfl_xor_sync(0xFFFFFFFFu, v.y, o);
          v.z += __shfl_xor_sync(0xFFFFFFFFu, v.z, o);
        }
        s2 = v.x;
        sa = v.y;
        sb = v.z;
      }
      buf ^= 1;  // two buffers: a warp can be at most one barrier ahead of another's reads
      if (active) {
        const float c2 = s2 * inv_d;
        const float c1 = post ? fmaf(-r2 * c2, sb, sa) * inv_d : 0.0f;  // no norm: dy = du
        const float2 r1v = splat2(r1), r2v = splat2(r2), k2 = splat2(-r2 * r2 * c2), k1 = splat2(-r1 * c1),
                     scale = splat2(a.res_scale);
        const long long at = static_cast<long long>(row) * a.nv + first_vec;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
          const int i = tr + k * TPR;
          if (i >= my_vecs) continue;
          float2 h[2], y[2], dh[2], dy[2];
          staged22<!HF>(staged + y_bytes, i, h);
          staged22<YB>(staged, i, y);
          staged22<!HF>(s_dh, i & dh_mask, dh);
          const uint2 gt = s_gate[i & gate_mask];
          const uint32_t pw[2] = {gpost[k].x, gpost[k].y}, tw[2] = {gt.x, gt.y};
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float2 d = fma2(h[j], k2, fma2(r2v, t[k][j], dh[j]));
            dh[j] = mul2(scale, d);
            const float2 du = mul2(unpack2(tw[j]), d), gp = unpack2(pw[j]), yh = mul2(y[j], r1v);
            acc_gate[k][j] = fma2(d, mul2(yh, gp), acc_gate[k][j]);
            acc_post[k][j] = fma2(du, yh, acc_post[k][j]);
            dy[j] = fma2(yh, k1, mul2(r1v, mul2(du, gp)));
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
    if (a.gate_out != nullptr && w.seg < a.segs) {
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        const int i = tr + k * TPR;
        if (i < my_vecs) {
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
  auto leave = [&](const float2 (&acc)[VPT][2], float4* part) {
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
  if (a.part_post != nullptr) leave(acc_post, a.part_post);
}

// out[g] = (accumulate ? out[g] : 0) + sum over p < parts of part[g * parts + p], column by column,
// in a fixed order.  Blocks of 16 vectors x 16 row lanes.
struct ColumnSum {
  const float4* part;
  float4* out;
  int groups, parts;
};

__global__ void __launch_bounds__(256) column_sum_kernel(const ColumnSum s0, const ColumnSum s1, const ColumnSum s2,
                                                         int nv, int chunks, int accumulate) {
  __shared__ float4 s_part[16][17];
  pdl::wait();
  int b = static_cast<int>(blockIdx.x) / chunks;
  const int chunk = static_cast<int>(blockIdx.x) - b * chunks;
  const ColumnSum* s = &s0;
  if (b >= s0.groups) {
    b -= s0.groups;
    s = &s1;
    if (b >= s1.groups) {
      b -= s1.groups;
      s = &s2;
    }
  }
  const int c = threadIdx.x & 15, rl = threadIdx.x >> 4;
  const int i = chunk * 16 + c;
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (i < nv) {
    const float4* p = s->part + static_cast<long long>(b) * s->parts * nv + i;
#pragma unroll 4
    for (int r = rl; r < s->parts; r += 16) {
      const float4 u = p[static_cast<long long>(r) * nv];
      v = make_float4(v.x + u.x, v.y + u.y, v.z + u.z, v.w + u.w);
    }
  }
  s_part[rl][c] = v;
  __syncthreads();
  if (rl == 0 && i < nv) {
    float4* out = s->out + static_cast<long long>(b) * nv + i;
#pragma unroll
    for (int r = 1; r < 16; ++r) {
      const float4 u = s_part[r][c];
      v = make_float4(v.x + u.x, v.y + u.y, v.z + u.z, v.w + u.w);
    }
    if (accumulate) {
      const float4 o = *out;
      v = make_float4(o.x + v.x, o.y + v.y, o.z + v.z, o.w + v.w);
    }
    *out = v;
  }
}

// Row lanes of the whole grid at most, over the shapes that a width can take.
int max_units(int d, int sms) {
  if (d <= 256) return 16 * sms;
  if (d <= 512) return 8 * sms;
  if (d <= 1024) return 4 * sms;
  if (d <= 2048) return 2 * sms;
  if (d <= 4096) return 2 * sms;
  return sms;
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

struct GradOut {
  float4* ws;
  float* dgate;
  bool pre, post;
  int accumulate;
};

template <int TPR, int VPT, int CS, bool YB, bool HF>
cudaError_t run_typed(BwdArgs& a, const GradOut& g, int& blocks, cudaStream_t stream, int num_sms) {
  constexpr int THREADS = bb_threads(TPR), RPB = THREADS / TPR, RING = bb_ring_bytes(TPR);
  auto kern = block_norm_bwd_kernel<TPR, VPT, CS, YB, HF>;
  const int smem_max = RING + 64;
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
  a.depth = std::max(1, std::min(kBbMaxDepth, (RING + 64) / (RPB * (a.slot_bytes + 8))));
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

template <int TPR, int VPT, int CS>
cudaError_t run(BwdArgs& a, const GradOut& g, bool yb, bool hf, int& blocks, cudaStream_t stream, int num_sms) {
  if (yb)
    return hf ? run_typed<TPR, VPT, CS, true, true>(a, g, blocks, stream, num_sms)
              : run_typed<TPR, VPT, CS, true, false>(a, g, blocks, stream, num_sms);
  return hf ? run_typed<TPR, VPT, CS, false, true>(a, g, blocks, stream, num_sms)
            : run_typed<TPR, VPT, CS, false, false>(a, g, blocks, stream, num_sms);
}

}  // namespace

// Partial rows: one per block for each gain, and one per segment for the gate (at most kBbWaves
// segments per row lane when a group of tokens is cut into several).
size_t block_norm_bwd_workspace_bytes(int d) {
  const size_t units = static_cast<size_t>(max_units(d, kBbMaxSms));
  return (2 + kBbWaves) * units * static_cast<size_t>(d) * sizeof(float);
}

cudaError_t launch_block_norm_bwd(const BlockNormBwdDev& p, cudaStream_t stream, int num_sms, uint32_t* err) {
  const int nv = p.d / 4;
  cudaError_t e = cudaSuccess;
  if (p.T == 0) {
    // the sums over no tokens (there are no gate rows either)
    if (!p.accumulate && p.dg_pre != nullptr) e = cudaMemsetAsync(p.dg_pre, 0, sizeof(float) * p.d, stream);
    if (e == cudaSuccess && !p.accumulate && p.dg_post != nullptr)
      e = cudaMemsetAsync(p.dg_post, 0, sizeof(float) * p.d, stream);
    return e;
  }
  if (num_sms > kBbMaxSms) num_sms = kBbMaxSms;
  BwdArgs a{};
  for (int q = 0; q < p.readers; ++q) a.dXn[q] = p.dXn[q];
  a.readers = p.readers;
  a.dH_in = p.dH_out;
  a.Y = p.Y;
  a.H = p.H_out;
  a.g_post = static_cast<const uint2*>(p.g_post);
  a.gate = static_cast<const uint2*>(p.gate);
  a.g_pre = static_cast<const uint2*>(p.g_pre);
  a.rstd = p.rstd;
  a.dY = static_cast<uint2*>(p.dY);
  a.dH = p.dH;
  a.res_scale = p.res_scale;
  a.T = p.T;
  a.nv = nv;
  a.err = err;
  a.period = p.gate != nullptr && p.gate_period < p.T ? p.gate_period : p.T;
  a.col_bytes = (p.y_bf16 ? 2 : 4) + (p.h_f32 ? 4 : 2) * (p.dH_out != nullptr ? 2 : 1) + 4 * p.readers +
                (p.gate != nullptr ? 2 : 0);
  const GradOut g{static_cast<float4*>(p.workspace), p.dgate, p.dg_pre != nullptr, p.dg_post != nullptr, p.accumulate};
  // 16 columns per thread where two rows can be staged for every row lane, else 8
  const bool yb = p.y_bf16, hf = p.h_f32, wide = a.col_bytes <= 13;
  const int d = p.d;
  int blocks = 0;
  if (d <= 256) e = run<32, 2, 1>(a, g, yb, hf, blocks, stream, num_sms);
  else if (d <= 512) e = run<64, 2, 1>(a, g, yb, hf, blocks, stream, num_sms);
  else if (d <= 1024) e = run<128, 2, 1>(a, g, yb, hf, blocks, stream, num_sms);
  else if (d <= 2048) e = run<256, 2, 1>(a, g, yb, hf, blocks, stream, num_sms);
  else if (d <= 4096) e = wide ? run<256, 4, 1>(a, g, yb, hf, blocks, stream, num_sms) : run<512, 2, 1>(a, g, yb, hf, blocks, stream, num_sms);
  else if (d <= 8192) e = wide ? run<512, 4, 1>(a, g, yb, hf, blocks, stream, num_sms) : run<512, 2, 2>(a, g, yb, hf, blocks, stream, num_sms);
  else e = wide ? run<512, 4, 2>(a, g, yb, hf, blocks, stream, num_sms) : run<512, 2, 4>(a, g, yb, hf, blocks, stream, num_sms);
  if (e != cudaSuccess) return e;
  const int groups = (p.T + a.period - 1) / a.period;
  ColumnSum pre{a.part_pre, reinterpret_cast<float4*>(p.dg_pre), p.dg_pre != nullptr ? 1 : 0, blocks};
  ColumnSum post{a.part_post, reinterpret_cast<float4*>(p.dg_post), p.dg_post != nullptr ? 1 : 0, blocks};
  ColumnSum gate{a.gate_out, reinterpret_cast<float4*>(p.dgate),
                 p.dgate != nullptr && a.segs_per_group > 1 ? groups : 0, a.segs_per_group};
  const int rows = pre.groups + post.groups + gate.groups;
  if (rows == 0) return cudaSuccess;
  const int chunks = (nv + 15) / 16;
  return pdl::launch(column_sum_kernel, rows * chunks, 256, 0, 1, stream, pre, post, gate, nv, chunks, p.accumulate);
}

}  // namespace sbl
