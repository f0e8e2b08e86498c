// Joining the pieces of the items that cross span boundaries, and the launch
// helpers of the kernels that make them.
#pragma once
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "paged_plan.cuh"

namespace attn {

// Merges the pieces of the items that cross span boundaries: block x looks at
// what worker x left and, where an item begins there and goes on, merges that
// item's rows (blockIdx.y of gridDim.y takes its part of them).  Few pieces:
// one warp a row.  Many (a long sequence alone in the batch): the block's
// warps share a row's pieces and add their sums.  Pieces are added in the
// order of their keys, so results do not vary from run to run.
// PACKED: rows stand as they are counted; else 128 / G whole tokens to each
// 128 rows.
template <int D, int TILE_ROWS, bool PACKED>
__global__ void __launch_bounds__(256) paged_join_kernel(const PagedParams p) {
  constexpr int NW = 8, V = D / 32;
  __shared__ float red[NW][D + 4];
  // every block waits, those without work too: what follows on the stream
  // relies on this grid's end for the end of the one before it
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Cut cut = p.cuts[blockIdx.x];
  if (cut.rows == 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, np = cut.np;
  const int per128 = PACKED ? 128 : 128 / p.G * p.G;
  auto place = [&](int i, int r) -> long long {
    return ((static_cast<long long>(blockIdx.x) + i) * 2 + (i == 0 ? cut.slot0 : 0)) * TILE_ROWS +
           (PACKED ? r : r + r / per128 * (128 - per128));
  };
  auto finish = [&](int r, float m, float l, const float (&acc)[V]) {
    const int x = cut.x0 + r, t = x / p.G, head = cut.h * p.G + x - t * p.G;
    const long long row = static_cast<long long>(cut.q0 + t) * p.hq + head;
    const long long li = static_cast<long long>(head) * p.n_tokens + cut.q0 + t;
    float fo, fi, lse;
    row_final(m, l, p.init_lse ? p.init_lse[li] : -INFINITY, fo, fi, lse);
#pragma unroll
    for (int c = 0; c < V; c += 2) store_pair<D>(p, row, lane * V + c, acc[c], acc[c + 1], fo, fi);
    if (lane == 0) p.lse[li] = lse;
  };
  // pieces i0, i0 + step, ... of row r summed by one warp
  auto gather = [&](int r, int i0, int step, float &m, float &l, float (&acc)[V]) {
    m = -INFINITY;
    for (int i = i0 + lane * step; i < np; i += 32 * step) m = fmaxf(m, p.part_ml[place(i, r) * 2]);
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    l = 0.f;
#pragma unroll
    for (int c = 0; c < V; ++c) acc[c] = 0.f;
    const float mb = m == -INFINITY ? 0.f : m;
    for (int base = i0; base < np; base += 32 * step) {
      float f = 0.f;
      if (base + lane * step < np) {
        const float2 ml = *reinterpret_cast<const float2 *>(p.part_ml + place(base + lane * step, r) * 2);
        f = exp2f(ml.x - mb);
        l += f * ml.y;
      }
      const int k1 = min(32, (np - base + step - 1) / step);
#pragma unroll 8
      for (int k = 0; k < k1; ++k) {
        const float g = __shfl_sync(0xffffffffu, f, k);
        const float *src = p.part_o + place(base + k * step, r) * D + lane * V;
        if constexpr (V == 4) {
          const float4 y = *reinterpret_cast<const float4 *>(src);
          acc[0] = fmaf(g, y.x, acc[0]);
          acc[1] = fmaf(g, y.y, acc[1]);
          acc[2] = fmaf(g, y.z, acc[2]);
          acc[3] = fmaf(g, y.w, acc[3]);
        } else {
          const float2 y = *reinterpret_cast<const float2 *>(src);
          acc[0] = fmaf(g, y.x, acc[0]);
          acc[1] = fmaf(g, y.y, acc[1]);
        }
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  };
  float m, l, acc[V];
  if (np <= NW) {
    for (int r = blockIdx.y * NW + warp; r < cut.rows; r += gridDim.y * NW) {
      gather(r, 0, 1, m, l, acc);
      finish(r, m, l, acc);
    }
    return;
  }
  for (int r = blockIdx.y; r < cut.rows; r += gridDim.y) {
    gather(r, warp, NW, m, l, acc);
#pragma unroll
    for (int c = 0; c < V; ++c) red[warp][lane * V + c] = acc[c];
    if (lane == 0) {
      red[warp][D] = m;
      red[warp][D + 1] = l;
    }
    __syncthreads();
    if (warp == 0) {
      float mt = -INFINITY, lt = 0.f;
#pragma unroll
      for (int k = 0; k < NW; ++k) mt = fmaxf(mt, red[k][D]);
      const float mb = mt == -INFINITY ? 0.f : mt;
#pragma unroll
      for (int c = 0; c < V; ++c) acc[c] = 0.f;
#pragma unroll
      for (int k = 0; k < NW; ++k) {
        const float f = exp2f(red[k][D] - mb);
        lt += f * red[k][D + 1];
#pragma unroll
        for (int c = 0; c < V; ++c) acc[c] = fmaf(f, red[k][lane * V + c], acc[c]);
      }
      finish(r, mt, lt, acc);
    }
    __syncthreads();
  }
}

template <typename K>
inline int raise_smem(K kern, size_t bytes, bool *done) {
  if (*done) return ATTN_OK;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes)) != cudaSuccess)
    return ATTN_ERR_CUDA;
  *done = true;
  return ATTN_OK;
}

// A launch that may start while the one before it on the stream drains; it
// waits for that one's memory before it reads any of it.
template <typename... A>
inline int launch_after(void (*kern)(A...), dim3 grid, int threads, size_t smem, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

constexpr size_t kSmemMax = 232448;



}  // namespace attn
