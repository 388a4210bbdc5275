// grad_group.cu -- the global gradient norm over many tensors, and clipping by it, on sm_100a.
//
// Sparse-BitNet summary ("Sparse-BitNet：1.58-bit 大模型天然兼容半结构化稀疏"), 方法步骤详情:
// the gradients are clipped to a global norm of 1.0 before the AdamW update.
//   S = sum over every tensor of g^2 (each square exact in fp64, sums in fp64),
//   norm = fl32(sqrt(S)),  c = fl32(min(1, max_norm / (sqrt(S) + 1e-6))) in fp64,
//   out = T_rn(fl32(g * c)).
//
// HBM bound.  c is known only after every gradient has been read, so clipping reads them twice
// and writes them once, where the floor is one read and one write.  Two launches: the first
// leaves one fp64 partial sum per block, the second sums the partials (every block, in the
// same order, so no block waits for another) and scales.  The scaling pass walks the tiles
// backwards, so it starts with what the norm pass read last and left in L2; gradients that fit
// there are read from HBM once.  No atomics: S is the same bits for the same tensors on every run on
// one device.  More than 128 tensors take several tables, a launch each: both passes go through the tables
// forwards, and backwards only within one, so there the scaling pass starts with the table that was
// read first and finds little of it in L2.
// Measured: norm pass alone 173 us for 1233 MB (7.1 TB/s), with clipping 550 us, where
// reading all but 64 MB twice and writing once takes 555 us at the measured copy rate.  Whole models, bf16, out of
// place: 716 MB in 216 tensors 339 us (two reads and a write at the copy rate 328), 5549 MB in 324 tensors
// 2518 us (2542); 418 MB in 126 tensors, one table, 190 us (191).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "pdl.cuh"
#include "sbl_internal.h"

namespace sbl {
namespace {

constexpr int kGgThreads = 256;
constexpr int kGgVecs = 4;                            // 16-byte vectors per thread and tile
constexpr int kGgTileVecs = kGgThreads * kGgVecs;     // 16 KB per tile
// The scaling pass is to find this much of the norm pass's last reads in L2 (of each table's, where there are
// several); what is read before goes first.  Measured on gradients of 308 MB: 144.5 us, with 32 or 128 MB 147.6, with plain loads 152.5
// (136.8 with the scaling pass as it is now).
constexpr unsigned kGgKeepTiles = (64u << 20) / (kGgTileVecs * 16);
constexpr int kGgTensors = 128;                       // tensors per launch (the table is a kernel parameter)

struct GradTable {
  const void* g[kGgTensors];
  void* out[kGgTensors];
  unsigned long long n[kGgTensors];
  unsigned int tile_start[kGgTensors + 1];
  unsigned int bf16[kGgTensors / 32];  // bit set: the tensor holds bf16
  int count;
  int in_place;  // every out is its g
};

// L2 eviction priorities: normal for what the scaling pass reads first, `first` for the rest (not
// evict_last: below the limit nothing reads those lines again, and they would stay).
__device__ __forceinline__ uint64_t policy_normal() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ uint64_t policy_first() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ uint4 load_hint(const uint4* p, uint64_t pol) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.L2::cache_hint.v4.u32 {%0, %1, %2, %3}, [%4], %5;"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p), "l"(pol));
  return v;
}
__device__ __forceinline__ void store_hint(uint4* p, const uint4& v, uint64_t pol) {
  asm volatile("st.global.L1::no_allocate.L2::cache_hint.v4.u32 [%0], {%1, %2, %3, %4}, %5;" ::"l"(p), "r"(v.x),
               "r"(v.y), "r"(v.z), "r"(v.w), "l"(pol)
               : "memory");
}

__device__ __forceinline__ double sq_add(float x, double s) {
  const double d = static_cast<double>(x);
  return fma(d, d, s);
}

// Sum over the block; every thread returns it (fixed order).
__device__ __forceinline__ double block_sum(double s, double* scratch) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = s;
  __syncthreads();
  double t = scratch[0];
#pragma unroll
  for (int w = 1; w < kGgThreads / 32; ++w) t += scratch[w];
  return t;
}

// Tile `t` of the table: its tensor, and the position of the tile's first vector in it.
struct TileCursor {
  int p;
  __device__ __forceinline__ void seek(const GradTable& tab, unsigned t) {
    while (t >= tab.tile_start[p + 1]) ++p;
  }
  __device__ __forceinline__ void seek_back(const GradTable& tab, unsigned t) {
    while (t < tab.tile_start[p]) --p;
  }
};

template <bool kBf16>
__device__ __forceinline__ double tile_sumsq(const void* g, unsigned long long n, unsigned long long v0, double s, uint64_t pol) {
  constexpr int PER = kBf16 ? 8 : 4;  // elements per vector
  const unsigned long long nv = n / PER;
  const uint4* gv = static_cast<const uint4*>(g);
  uint4 v[kGgVecs];
#pragma unroll
  for (int k = 0; k < kGgVecs; ++k) {
    const unsigned long long i = v0 + k * kGgThreads + threadIdx.x;
    v[k] = i < nv ? load_hint(gv + i, pol) : make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int k = 0; k < kGgVecs; ++k) {
    const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (kBf16) {
        s = sq_add(__uint_as_float(w[j] << 16), s);
        s = sq_add(__uint_as_float(w[j] & 0xFFFF0000u), s);
      } else {
        s = sq_add(__uint_as_float(w[j]), s);
      }
    }
  }
  // the n % PER elements behind the last whole vector belong to the tile that vector nv would be in
  if (v0 <= nv && nv < v0 + kGgTileVecs) {
    const unsigned long long e = nv * PER + threadIdx.x;
    if (threadIdx.x < PER && e < n) {
      if constexpr (kBf16) {
        s = sq_add(__uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(g)[e]) << 16), s);
      } else {
        s = sq_add(static_cast<const float*>(g)[e], s);
      }
    }
  }
  return s;
}

// keep: tiles at the end of the table that L2 should hold until the scaling pass.
__global__ void __launch_bounds__(kGgThreads) grad_sumsq_kernel(const __grid_constant__ GradTable tab,
                                                                double* partial, unsigned keep) {
  __shared__ double scratch[kGgThreads / 32];
  pdl::wait();
  pdl::release();
  const unsigned total = tab.tile_start[tab.count];
  const uint64_t normal = policy_normal(), first = policy_first();
  double s = 0.0;
  TileCursor c{0};
  for (unsigned t = blockIdx.x; t < total; t += gridDim.x) {
    c.seek(tab, t);
    const unsigned long long v0 = static_cast<unsigned long long>(t - tab.tile_start[c.p]) * kGgTileVecs;
    const uint64_t pol = total - t <= keep ? normal : first;
    s = ((tab.bf16[c.p >> 5] >> (c.p & 31)) & 1u) ? tile_sumsq<true>(tab.g[c.p], tab.n[c.p], v0, s, pol)
                                                  : tile_sumsq<false>(tab.g[c.p], tab.n[c.p], v0, s, pol);
  }
  s = block_sum(s, scratch);
  if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

// S from the blocks' partial sums; every block that calls this gets the same bits.
__device__ __forceinline__ double total_sumsq(const double* partial, int count, double* scratch) {
  double s = 0.0;
  for (int i = threadIdx.x; i < count; i += kGgThreads) s += partial[i];
  return block_sum(s, scratch);
}

__device__ __forceinline__ float clip_factor(double S, double max_norm) {
  const double q = max_norm / (sqrt(S) + 1e-6);
  return q >= 1.0 ? 1.0f : static_cast<float>(q);  // a NaN norm gives a NaN factor
}

__device__ __forceinline__ void store_norm(double S, float c, double* sumsq, float* norm, float* clip) {
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    *sumsq = S;
    if (norm != nullptr) *norm = static_cast<float>(sqrt(S));
    if (clip != nullptr) *clip = c;
  }
}

__global__ void __launch_bounds__(kGgThreads) grad_norm_finish_kernel(const double* partial, int count,
                                                                      double* sumsq, float* norm) {
  __shared__ double scratch[kGgThreads / 32];
  pdl::wait();
  const double S = total_sumsq(partial, count, scratch);
  store_norm(S, 0.0f, sumsq, norm, nullptr);
}

template <bool kBf16>
__device__ __forceinline__ void tile_scale(const void* g, void* out, unsigned long long n, unsigned long long v0,
                                           float c) {
  const uint64_t first = policy_first();
  constexpr int PER = kBf16 ? 8 : 4;
  const unsigned long long nv = n / PER;
  const uint4* gv = static_cast<const uint4*>(g);
  uint4* ov = static_cast<uint4*>(out);
  uint4 v[kGgVecs];
#pragma unroll
  for (int k = 0; k < kGgVecs; ++k) {
    const unsigned long long i = v0 + k * kGgThreads + threadIdx.x;
    v[k] = i < nv ? load_hint(gv + i, first) : make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int k = 0; k < kGgVecs; ++k) {
    const unsigned long long i = v0 + k * kGgThreads + threadIdx.x;
    uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (kBf16) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(__fmul_rn(__uint_as_float(w[j] << 16), c),
                                                       __fmul_rn(__uint_as_float(w[j] & 0xFFFF0000u), c));
        w[j] = *reinterpret_cast<const uint32_t*>(&p);
      } else {
        w[j] = __float_as_uint(__fmul_rn(__uint_as_float(w[j]), c));
      }
    }
    if (i < nv) store_hint(ov + i, make_uint4(w[0], w[1], w[2], w[3]), first);
  }
  if (v0 <= nv && nv < v0 + kGgTileVecs) {
    const unsigned long long e = nv * PER + threadIdx.x;
    if (threadIdx.x < PER && e < n) {
      if constexpr (kBf16) {
        const float x = __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(g)[e]) << 16);
        static_cast<__nv_bfloat16*>(out)[e] = __float2bfloat16_rn(__fmul_rn(x, c));
      } else {
        static_cast<float*>(out)[e] = __fmul_rn(static_cast<const float*>(g)[e], c);
      }
    }
  }
}

__global__ void __launch_bounds__(kGgThreads)
    grad_scale_kernel(const __grid_constant__ GradTable tab, const double* partial, int partials,
                      double max_norm, double* sumsq, float* norm, float* clip) {
  __shared__ double scratch[kGgThreads / 32];
  pdl::wait();
  const double S = total_sumsq(partial, partials, scratch);
  const float c = clip_factor(S, max_norm);
  if (sumsq != nullptr) store_norm(S, c, sumsq, norm, clip);
  const unsigned total = tab.tile_start[tab.count];
  if (blockIdx.x >= total || (c == 1.0f && tab.in_place != 0)) return;  // in place, below the limit: nothing to do
  TileCursor cur{tab.count - 1};
  for (unsigned u = blockIdx.x; u < total; u += gridDim.x) {
    const unsigned t = total - 1 - u;
    cur.seek_back(tab, t);
    const int p = cur.p;
    if (c == 1.0f && tab.out[p] == tab.g[p]) continue;
    const unsigned long long v0 = static_cast<unsigned long long>(t - tab.tile_start[p]) * kGgTileVecs;
    if ((tab.bf16[p >> 5] >> (p & 31)) & 1u)
      tile_scale<true>(tab.g[p], tab.out[p], tab.n[p], v0, c);
    else
      tile_scale<false>(tab.g[p], tab.out[p], tab.n[p], v0, c);
  }
}

constexpr int kGgBlocksPerSm = 4;
// Tiles per block of the scaling pass.  Blocks that come one after the other walk the memory more evenly
// than four per SM that stay: 1233 MB 550 us against 593 (6.4 against 5.7 TB/s of that pass); a block
// reads the partial sums (in L2, 5 KB for each table of up to 128 tensors) for two tiles.  In place the blocks stay: below the limit there
// is nothing to scale, and 38000 blocks that find that out take 50 us, 592 take 3.
constexpr unsigned kGgScaleTiles = 2;
constexpr int kGgMaxBlocks = 1024;  // of one launch: sizes the workspace

int gg_blocks(int num_sms) {
  return num_sms * kGgBlocksPerSm < kGgMaxBlocks ? num_sms * kGgBlocksPerSm : kGgMaxBlocks;
}

// Fills the table with up to kGgTensors tensors from `i`; returns the index behind the last.
int fill_table(const GradTensorDev* t, int i, int count, GradTable& tab) {
  tab.count = 0;
  tab.in_place = 1;
  tab.tile_start[0] = 0;
  for (int k = 0; k < kGgTensors / 32; ++k) tab.bf16[k] = 0u;
  unsigned long long tiles = 0;
  for (; i < count && tab.count < kGgTensors; ++i) {
    if (t[i].n == 0) continue;
    const unsigned long long per_tile = static_cast<unsigned long long>(kGgTileVecs) * (t[i].bf16 ? 8 : 4);
    const unsigned long long mine = (t[i].n + per_tile - 1) / per_tile;
    if (tab.count > 0 && tiles + mine > 0x7FFFFFFFull) break;
    const int p = tab.count++;
    tab.g[p] = t[i].g;
    tab.out[p] = t[i].out;
    if (t[i].out != t[i].g) tab.in_place = 0;
    tab.n[p] = t[i].n;
    if (t[i].bf16) tab.bf16[p >> 5] |= 1u << (p & 31);
    tiles += mine;
    tab.tile_start[p + 1] = static_cast<unsigned>(tiles);
  }
  return i;
}

}  // namespace

// One row of partial sums per launch of the norm pass; launches are cut by tensor count (and by
// a tile count that no memory of this device reaches).
size_t grad_group_workspace_bytes(int count) {
  const size_t launches = count <= 0 ? 1 : (static_cast<size_t>(count) + kGgTensors - 1) / kGgTensors;
  return (launches + 1) * kGgMaxBlocks * sizeof(double);
}

cudaError_t launch_grad_group(const GradTensorDev* t, int count, bool clip_them, double max_norm, double* sumsq,
                              float* norm, float* clip, void* workspace, cudaStream_t stream, int num_sms) {
  double* partial = static_cast<double*>(workspace);
  int used = 0;
  GradTable tab;
  for (int i = 0; i < count;) {
    i = fill_table(t, i, count, tab);
    if (tab.count == 0) break;
    const unsigned total = tab.tile_start[tab.count];
    const int grid = static_cast<int>(total < static_cast<unsigned>(gg_blocks(num_sms)) ? total : gg_blocks(num_sms));
    const cudaError_t e = pdl::launch(grad_sumsq_kernel, grid, kGgThreads, 0, 1, stream, tab, partial + used,
                                    clip_them ? kGgKeepTiles : 0u);
    if (e != cudaSuccess) return e;
    used += grid;
  }
  if (!clip_them || used == 0) {
    // nothing to scale: S (0 for no elements) and the norm; with clipping the factor too
    if (clip_them) {
      tab.count = 0;
      tab.tile_start[0] = 0;
      return pdl::launch(grad_scale_kernel, 1, kGgThreads, 0, 1, stream, tab, static_cast<const double*>(partial), used, max_norm, sumsq,
                       norm, clip);
    }
    return pdl::launch(grad_norm_finish_kernel, 1, kGgThreads, 0, 1, stream, static_cast<const double*>(partial), used, sumsq, norm);
  }
  bool first = true;
  for (int i = 0; i < count;) {
    i = fill_table(t, i, count, tab);
    if (tab.count == 0) break;
    const unsigned total = tab.tile_start[tab.count];
    const unsigned blocks = (total + kGgScaleTiles - 1) / kGgScaleTiles;
    const unsigned stay = static_cast<unsigned>(gg_blocks(num_sms));
    const int grid = static_cast<int>(tab.in_place != 0 && blocks > stay ? stay : blocks);
    const cudaError_t e = pdl::launch(grad_scale_kernel, grid, kGgThreads, 0, 1, stream, tab, static_cast<const double*>(partial), used,
                                    max_norm, first ? sumsq : static_cast<double*>(nullptr), norm, clip);
    if (e != cudaSuccess) return e;
    first = false;
  }
  return cudaSuccess;
}

}  // namespace sbl
