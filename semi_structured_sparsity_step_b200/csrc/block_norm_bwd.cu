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
// HBM bound: one read of each dX, dH, y and h', one write of dy and dh.  TPR threads share a row,
// 8 columns each (2048 columns per block; wider rows go to a cluster of CS blocks that exchange the
// three sums through distributed shared memory).  A thread keeps its columns for all its rows, so
// the column sums stay in registers.  The rows to come are staged in a ring in shared memory by
// bulk copies, one ring per row lane; a slot is refilled once its row's sums have met.  Column sums leave as one partial row per block (dgate: per segment of rows
// with one gate row), and a second launch adds the partial rows in a fixed order: no atomics.
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

constexpr int kBbThreads = 256;
constexpr int kBbVpt = 2;            // vectors of 4 columns per thread
constexpr int kBbBlocksPerSm = 2;
constexpr int kBbMaxSms = 160;       // sizes the workspace
constexpr int kBbWaves = 4;          // segments per row lane at most

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
  int depth, slot_bytes; // rows of the ring, bytes of a staged row (at most)
  uint32_t* err;
};

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
  return x;
}

template <int TPR, int CS, bool YB, bool HF>
__global__ void __launch_bounds__(kBbThreads, kBbBlocksPerSm) block_norm_bwd_kernel(const BwdArgs a) {
  constexpr int RPB = kBbThreads / TPR;
  constexpr int WPR = TPR / 32;
  constexpr int SLOTS = CS > 1 ? CS * 8 : 8;
  __shared__ float4 s_sum[2][SLOTS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rib = threadIdx.x / TPR;
  const int tr = threadIdx.x % TPR;
  const int rank = CS > 1 ? static_cast<int>(pair::cluster_rank()) : 0;
  const int unit = static_cast<int>(blockIdx.x) / CS * RPB + rib;  // row lane
  const int units = static_cast<int>(gridDim.x) / CS * RPB;
  const int v0 = rank * a.vecs_per_cta + tr;
  const int v1 = min(a.nv, (rank + 1) * a.vecs_per_cta);
  const bool post = a.g_post != nullptr;
  const float inv_d = 1.0f / (4.0f * static_cast<float>(a.nv));
  // one staged row: y, h', dH (if given), the readers' gradients, the gate row (if given)
  const int cols = (v1 - rank * a.vecs_per_cta) * 4;
  const uint32_t b16 = static_cast<uint32_t>(cols > 0 ? cols : 0) * 2u, b32 = 2u * b16;
  const uint32_t y_bytes = YB ? b16 : b32, h_bytes = HF ? b32 : b16;
  const uint32_t off_dh = y_bytes + h_bytes;
  const uint32_t off_dx = off_dh + (a.dH_in != nullptr ? h_bytes : 0u);
  const uint32_t off_gate = off_dx + static_cast<uint32_t>(a.readers) * b32;
  const uint32_t row_bytes = off_gate + (a.gate != nullptr ? b16 : 0u);
  extern __shared__ __align__(128) uint8_t ring[];
  uint8_t* slots = ring + static_cast<size_t>(rib) * a.depth * a.slot_bytes;
  uint64_t* bars =
      reinterpret_cast<uint64_t*>(ring + static_cast<size_t>(RPB) * a.depth * a.slot_bytes) + rib * a.depth;
  __shared__ int s_abort;
  if (tr == 0) {
    for (int i = 0; i < a.depth; ++i) mbar_init(&bars[i], 1);
    s_abort = 0;
    fence_mbar_init();
  }
  auto request = [&](int row, int slot) {
    uint8_t* dst = slots + static_cast<size_t>(slot) * a.slot_bytes;
    uint64_t* bar = &bars[slot];
    const long long at = static_cast<long long>(row) * a.nv * 4 + rank * a.vecs_per_cta * 4;
    mbar_arrive_expect_tx(bar, row_bytes);
    bulk_load(dst, static_cast<const uint8_t*>(a.Y) + at * (YB ? 2 : 4), y_bytes, bar);
    bulk_load(dst + y_bytes, static_cast<const uint8_t*>(a.H) + at * (HF ? 4 : 2), h_bytes, bar);
    if (a.dH_in != nullptr)
      bulk_load(dst + off_dh, static_cast<const uint8_t*>(a.dH_in) + at * (HF ? 4 : 2), h_bytes, bar);
    for (int q = 0; q < a.readers; ++q) bulk_load(dst + off_dx + q * b32, a.dXn[q] + at, b32, bar);
    if (a.gate != nullptr) {
      const long long gat = static_cast<long long>(row / a.period) * a.nv * 4 + rank * a.vecs_per_cta * 4;
      bulk_load(dst + off_gate, reinterpret_cast<const uint8_t*>(a.gate) + gat * 2, b16, bar);
    }
  };
  __syncthreads();
  if constexpr (CS > 1) pair::cluster_sync();  // every block of the cluster is there
  pdl::wait();

  uint2 gpre[kBbVpt], gpost[kBbVpt];
  float acc_pre[kBbVpt][4], acc_post[kBbVpt][4], acc_gate[kBbVpt][4];
#pragma unroll
  for (int k = 0; k < kBbVpt; ++k) {
    const int i = v0 + k * TPR;
    gpre[k] = gpost[k] = make_uint2(0x3F803F80u, 0x3F803F80u);
    if (i < v1) {
      gpre[k] = __ldg(a.g_pre + i);
      if (post) gpost[k] = __ldg(a.g_post + i);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) acc_pre[k][j] = acc_post[k][j] = acc_gate[k][j] = 0.0f;
  }

  // Every row lane walks its segments, seg_rows steps each (steps past the segment's rows are
  // inactive), so all lanes of a block or cluster take the same number of steps and barriers.
  const int rounds = (a.segs + units - 1) / units;
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
  enter(ahead);
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
  if (tr == 0 && cols > 0)
    for (int i = 0; i < a.depth; ++i) request_next();

  int buf = 0;
  for (int rd = 0; rd < rounds; ++rd) {
    const int seg = w.seg;
    for (int step = 0; step < a.seg_rows; ++step) {
      const bool cur_active = step < w.rows;
      const int cur_row = w.row + step;
      float cur_r1 = 0.0f, cur_r2 = 0.0f;
      if (cur_active) {
        cur_r1 = __ldg(a.rstd + cur_row);
        cur_r2 = __ldg(a.rstd + a.T + cur_row);
      }
      const uint8_t* staged = slots + static_cast<size_t>(pos.slot) * a.slot_bytes;
      if (cur_active && cols > 0) {
        mbar_wait(&bars[pos.slot], pos.parity, &s_abort, a.err);
        pos.next(a.depth);
      }
      float t[kBbVpt][4], xh[kBbVpt][4], dhin[kBbVpt][4], yh[kBbVpt][4];
      uint2 gt[kBbVpt];
      float s2 = 0.0f, sa = 0.0f, sb = 0.0f;
#pragma unroll
      for (int k = 0; k < kBbVpt; ++k) {
        const int i = tr + k * TPR;
        gt[k] = make_uint2(0x3F803F80u, 0x3F803F80u);  // 1.0
        float dx[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) xh[k][j] = dhin[k][j] = yh[k][j] = dx[j] = 0.0f;
        if (cur_active && v0 + k * TPR < v1) {
          staged4<YB>(staged, i, yh[k]);
          staged4<!HF>(staged + y_bytes, i, xh[k]);
          if (a.dH_in != nullptr) staged4<!HF>(staged + off_dh, i, dhin[k]);
          staged4<false>(staged + off_dx, i, dx);
          for (int q = 1; q < a.readers; ++q) {
            float more[4];
            staged4<false>(staged + off_dx + q * b32, i, more);
#pragma unroll
            for (int j = 0; j < 4; ++j) dx[j] += more[j];
          }
          if (a.gate != nullptr) gt[k] = reinterpret_cast<const uint2*>(staged + off_gate)[i];
        }
        float g[4], gp[4], gg[4];
        unpack4(gpre[k], g);
        unpack4(gpost[k], gp);
        unpack4(gt[k], gg);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          xh[k][j] *= cur_r2;
          acc_pre[k][j] = fmaf(dx[j], xh[k][j], acc_pre[k][j]);
          t[k][j] = dx[j] * g[j];
          s2 = fmaf(t[k][j], xh[k][j], s2);
          if (post) {
            yh[k][j] *= cur_r1;
            const float wt = gg[j] * gp[j] * yh[k][j];
            sa = fmaf(wt, fmaf(cur_r2, t[k][j], dhin[k][j]), sa);
            sb = fmaf(wt, xh[k][j], sb);
          }
        }
      }
      s2 = warp_sum(s2);
      if (post) {
        sa = warp_sum(sa);
        sb = warp_sum(sb);
      }
      if constexpr (CS > 1) {
        if (lane < CS) {
          const uint32_t dst = pair::map_to(smem_u32(&s_sum[buf][rank * 8 + warp]), static_cast<uint32_t>(lane));
          asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "f"(s2), "f"(sa), "f"(sb),
                       "f"(0.0f)
                       : "memory");
        }
        pair::cluster_sync();
        float4 v = s_sum[buf][lane % SLOTS];
        if (lane >= SLOTS) v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if constexpr (SLOTS > 32) {
          const float4 u = s_sum[buf][lane + 32];
          v.x += u.x;
          v.y += u.y;
          v.z += u.z;
        }
        s2 = warp_sum(v.x);
        if (post) {
          sa = warp_sum(v.y);
          sb = warp_sum(v.z);
        }
      } else if constexpr (WPR > 1) {
        if (lane == 0) s_sum[buf][warp] = make_float4(s2, sa, sb, 0.0f);
        lane_sync<TPR, kBbThreads>(rib);
        s2 = sa = sb = 0.0f;
#pragma unroll
        for (int w = 0; w < WPR; ++w) {
          const float4 v = s_sum[buf][rib * WPR + w];
          s2 += v.x;
          sa += v.y;
          sb += v.z;
        }
      } else {
        __syncwarp();
      }
      // every thread of the row lane is past its reads of the slot
      if (tr == 0 && cur_active && cols > 0) request_next();
      buf ^= 1;  // two buffers: a warp can be at most one barrier ahead of another's reads
      const float c2 = s2 * inv_d;
      const float c1 = fmaf(-cur_r2 * c2, sb, sa) * inv_d;
      const long long at = static_cast<long long>(cur_row) * a.nv;
#pragma unroll
      for (int k = 0; k < kBbVpt; ++k) {
        const int i = v0 + k * TPR;
        float gp[4], gg[4], dh[4], dy[4];
        unpack4(gpost[k], gp);
        unpack4(gt[k], gg);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float d = fmaf(cur_r2, fmaf(-xh[k][j], c2, t[k][j]), dhin[k][j]);
          dh[j] = a.res_scale * d;
          acc_gate[k][j] = fmaf(d, yh[k][j] * gp[j], acc_gate[k][j]);
          const float du = gg[j] * d;
          if (post) {
            acc_post[k][j] = fmaf(du, yh[k][j], acc_post[k][j]);
            dy[j] = cur_r1 * fmaf(-yh[k][j], c1, du * gp[j]);
          } else {
            dy[j] = du;
          }
        }
        if (cur_active && i < v1) {
          a.dY[at + i] = pack4(dy);
          if (a.dH != nullptr) store4<!HF>(a.dH, at + i, dh);
        }
      }
    }
    w.seg += units;
    enter(w);
    if (a.gate_out != nullptr && seg < a.segs) {
#pragma unroll
      for (int k = 0; k < kBbVpt; ++k) {
        const int i = v0 + k * TPR;
        if (i < v1) {
          float4* out = a.gate_out + static_cast<long long>(seg) * a.nv + i;
          float4 v = make_float4(acc_gate[k][0], acc_gate[k][1], acc_gate[k][2], acc_gate[k][3]);
          if (a.gate_accumulate) {
            const float4 o = *out;
            v = make_float4(o.x + v.x, o.y + v.y, o.z + v.z, o.w + v.w);
          }
          *out = v;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) acc_gate[k][j] = 0.0f;
      }
    }
  }

  // the block's row lanes meet in shared memory (the ring's, every staged row is consumed): one
  // partial row per block
  float4* s_col = reinterpret_cast<float4*>(ring);
  auto leave = [&](const float (&acc)[kBbVpt][4], float4* part) {
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kBbVpt; ++k)
      s_col[rib * (TPR * kBbVpt) + k * TPR + tr] = make_float4(acc[k][0], acc[k][1], acc[k][2], acc[k][3]);
    __syncthreads();
    for (int c = threadIdx.x; c < TPR * kBbVpt; c += kBbThreads) {
      const int i = rank * a.vecs_per_cta + c;
      if (i >= v1) continue;
      float4 s = s_col[c];
#pragma unroll
      for (int r = 1; r < RPB; ++r) {
        const float4 v = s_col[r * (TPR * kBbVpt) + c];
        s = make_float4(s.x + v.x, s.y + v.y, s.z + v.z, s.w + v.w);
      }
      part[static_cast<long long>(blockIdx.x / CS) * a.nv + i] = s;
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

// Threads per row (row lanes of a block) and blocks per row (cluster size) by width.
struct Shape {
  int tpr, cs;
};
Shape shape_of(int d) {
  if (d <= 256) return {32, 1};
  if (d <= 512) return {64, 1};
  if (d <= 1024) return {128, 1};
  if (d <= 2048) return {256, 1};
  if (d <= 4096) return {256, 2};
  if (d <= 8192) return {256, 4};
  return {256, 8};
}

int max_units(int d, int sms) {
  const Shape s = shape_of(d);
  return kBbBlocksPerSm * sms / s.cs * (kBbThreads / s.tpr);
}

constexpr int kBbRingBytes = 104 * 1024;  // per block, two blocks per SM
constexpr int kBbMaxDepth = 4;
constexpr int kBbColBytes = kBbThreads * kBbVpt * 16;  // the row lanes' column sums, at the end

template <int TPR, int CS, bool YB, bool HF>
cudaError_t run_typed(BwdArgs a, int grid, cudaStream_t stream) {
  constexpr int RPB = kBbThreads / TPR;
  a.slot_bytes = a.vecs_per_cta * 4 *
                 ((YB ? 2 : 4) + (HF ? 4 : 2) * (a.dH_in != nullptr ? 2 : 1) + 4 * a.readers + (a.gate != nullptr ? 2 : 0));
  a.depth = kBbRingBytes / (RPB * a.slot_bytes);
  if (a.depth > kBbMaxDepth) a.depth = kBbMaxDepth;
  if (a.depth < 1) a.depth = 1;
  int smem = RPB * a.depth * (a.slot_bytes + 8);
  if (smem < kBbColBytes) smem = kBbColBytes;
  auto kern = block_norm_bwd_kernel<TPR, CS, YB, HF>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kBbRingBytes + 1024);
  if (e != cudaSuccess) return e;
  return pdl::launch(kern, grid, kBbThreads, smem, CS, stream, a);
}

// How many clusters of CS blocks are resident at once: fewer than the SMs alone would hold, as a
// cluster stays within one group of SMs.  Asked once per device for the widest staged row.
template <int CS>
int resident_clusters(int num_sms) {
  static std::atomic<int> cached[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return num_sms / CS;
  int n = cached[dev].load();
  if (n == 0) {
    auto kern = block_norm_bwd_kernel<256, CS, false, true>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(CS);
    cfg.blockDim = dim3(kBbThreads);
    cfg.dynamicSmemBytes = kBbRingBytes + 1024;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = CS;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kBbRingBytes + 1024) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n < 1)
      n = num_sms / CS;
    if (n > kBbBlocksPerSm * num_sms / CS) n = kBbBlocksPerSm * num_sms / CS;
    cached[dev].store(n);
  }
  return n;
}

template <int TPR, int CS>
cudaError_t run(const BwdArgs& a, bool yb, bool hf, int grid, cudaStream_t stream) {
  if (yb) return hf ? run_typed<TPR, CS, true, true>(a, grid, stream) : run_typed<TPR, CS, true, false>(a, grid, stream);
  return hf ? run_typed<TPR, CS, false, true>(a, grid, stream) : run_typed<TPR, CS, false, false>(a, grid, stream);
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
  const Shape sh = shape_of(p.d);
  const int rpb = kBbThreads / sh.tpr;
  if (num_sms > kBbMaxSms) num_sms = kBbMaxSms;
  int units_max = max_units(p.d, num_sms);
  if (sh.cs == 2) units_max = std::min(units_max, resident_clusters<2>(num_sms));
  if (sh.cs == 4) units_max = std::min(units_max, resident_clusters<4>(num_sms));
  if (sh.cs == 8) units_max = std::min(units_max, resident_clusters<8>(num_sms));
  // Cut each group of tokens that share a gate row into segs_per_group segments: the choice with
  // the fewest steps on the busiest row lane, a segment's end counted as half a step.
  const bool gated = p.gate != nullptr;
  const int period = gated && p.gate_period < p.T ? p.gate_period : p.T;
  const int groups = (p.T + period - 1) / period;
  int seg_rows = period, per_group = 1;
  double best = 1e30;
  for (int w = 0; w <= kBbWaves; ++w) {
    long long s = w == 0 ? 1 : static_cast<long long>(w) * units_max / groups;
    if (s < 1) s = 1;
    if (s > period) s = period;
    const int rows = static_cast<int>((period + s - 1) / s);
    const int pg = (period + rows - 1) / rows;
    const long long segs = static_cast<long long>(groups) * pg;
    const double cost = static_cast<double>((segs + units_max - 1) / units_max) * (rows + (gated ? 0.5 : 0.0));
    if (cost < best) {
      best = cost;
      seg_rows = rows;
      per_group = pg;
    }
  }
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
  // a multiple of 16 columns, so that every block's slice of a row starts and ends on 16 bytes
  a.vecs_per_cta = sh.cs > 1 ? (nv / 4 + sh.cs - 1) / sh.cs * 4 : nv;
  a.err = err;
  a.period = period;
  a.seg_rows = seg_rows;
  a.segs_per_group = per_group;
  a.segs = groups * per_group;
  const int units = a.segs < units_max ? a.segs : units_max;
  const int blocks = (units + rpb - 1) / rpb;  // clusters, when a row takes one
  float4* ws = static_cast<float4*>(p.workspace);
  const size_t rows_max = static_cast<size_t>(units_max);
  if (p.dg_pre != nullptr) a.part_pre = ws;
  if (p.dg_post != nullptr) a.part_post = ws + rows_max * nv;
  float4* gate_part = ws + 2 * rows_max * nv;
  if (p.dgate != nullptr) {
    a.gate_out = per_group > 1 ? gate_part : reinterpret_cast<float4*>(p.dgate);
    a.gate_accumulate = per_group > 1 ? 0 : p.accumulate;
  }
  const int grid = blocks * sh.cs;
  switch (sh.tpr * 16 + sh.cs) {
    case 32 * 16 + 1: e = run<32, 1>(a, p.y_bf16, p.h_f32, grid, stream); break;
    case 64 * 16 + 1: e = run<64, 1>(a, p.y_bf16, p.h_f32, grid, stream); break;
    case 128 * 16 + 1: e = run<128, 1>(a, p.y_bf16, p.h_f32, grid, stream); break;
    case 256 * 16 + 1: e = run<256, 1>(a, p.y_bf16, p.h_f32, grid, stream); break;
    case 256 * 16 + 2: e = run<256, 2>(a, p.y_bf16, p.h_f32, grid, stream); break;
    case 256 * 16 + 4: e = run<256, 4>(a, p.y_bf16, p.h_f32, grid, stream); break;
    default: e = run<256, 8>(a, p.y_bf16, p.h_f32, grid, stream); break;
  }
  if (e != cudaSuccess) return e;
  ColumnSum pre{a.part_pre, reinterpret_cast<float4*>(p.dg_pre), p.dg_pre != nullptr ? 1 : 0, blocks};
  ColumnSum post{a.part_post, reinterpret_cast<float4*>(p.dg_post), p.dg_post != nullptr ? 1 : 0, blocks};
  ColumnSum gate{gate_part, reinterpret_cast<float4*>(p.dgate), p.dgate != nullptr && per_group > 1 ? groups : 0,
                 per_group};
  const int rows = pre.groups + post.groups + gate.groups;
  if (rows == 0) return cudaSuccess;
  const int chunks = (nv + 15) / 16;
  return pdl::launch(column_sum_kernel, rows * chunks, 256, 0, 1, stream, pre, post, gate, nv, chunks, p.accumulate);
}

}  // namespace sbl
