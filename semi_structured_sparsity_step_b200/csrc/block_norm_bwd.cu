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
// Measured: 32768 x 2048, three readers, a gate per sequence 255 us, 0.96 of the measured copy rate;
// 16384 x 2048, one reader, bf16, no gate 87 us (0.83); 4096 x 8192 with a gate 92 us (0.78), where the
// instructions per element (51) keep it from the memory's rate.
#include <cuda_runtime.h>
#include <cstdint>

#include "block_norm_bwd.cuh"

namespace sbl {
namespace {

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
  a.col_bytes = (p.g_post == nullptr && p.dgate == nullptr ? 0 : p.y_bf16 ? 2 : 4) +
                (p.h_f32 ? 4 : 2) * (p.dH_out != nullptr ? 2 : 1) + 4 * p.readers +
                (p.gate != nullptr ? 2 : 0);
  const GradOut g{static_cast<float4*>(p.workspace), p.dgate, p.dg_pre != nullptr, p.dg_post != nullptr, p.accumulate};
  int blocks = 0;
  const auto mode = p.g_post != nullptr ? (p.gate != nullptr ? block_norm_bwd_post_gate : block_norm_bwd_post)
                                        : (p.gate != nullptr ? block_norm_bwd_gate : block_norm_bwd_plain);
  e = mode(a, g, p.y_bf16, p.h_f32, blocks, stream, num_sms);
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
