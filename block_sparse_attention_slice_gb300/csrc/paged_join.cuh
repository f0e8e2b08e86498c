// Joining the pieces of the items that cross span boundaries, and the launch
// helpers of the kernels that make them.
#pragma once
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "paged_plan.cuh"

namespace attn {

// Merges the pieces of the items that cross span boundaries: block x looks at
// the boundary between spans x and x + 1 and, if it is the first inside an
// item, merges that item's rows (blockIdx.y of gridDim.y takes every
// gridDim.y-th).  Few pieces: one warp a row.  Many (a long sequence alone in
// the batch): the block's warps share a row's pieces and add their sums.
template <int D, int ROWS, int KL, int TILE_ROWS>
__global__ void __launch_bounds__(256) paged_join_kernel(const PagedParams p, int tpi) {
  constexpr int NW = 8, V = D / 32;
  extern __shared__ __align__(16) uint8_t join_smem[];
  long long *scan = reinterpret_cast<long long *>(join_smem);
  float *red = reinterpret_cast<float *>(join_smem + 80);          // [NW][D + 2]
  long long *first = reinterpret_cast<long long *>(join_smem + 80 + NW * (D + 4) * 4);
  SeqInfo *info = ROWS > 0 ? reinterpret_cast<SeqInfo *>(first + p.n_seqs + 1) : nullptr;
  make_plan<ROWS, KL, 256>(p, tpi, first, info, scan);
  // every block waits, those without work too: what follows on the stream
  // relies on this grid's end for the end of the one before it
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const long long total = first[p.n_seqs], span = span_of(p, total);
  const long long cut = (blockIdx.x + 1) * span;
  if (cut >= total) return;
  Walk<ROWS, KL> w;
  w.seek(p, first, info, tpi, cut);
  const long long f0 = cut - w.i, f1 = f0 + w.sp.n;
  if (w.i == 0 || f0 < cut - span) return;      // the cut lies between items, or is not the item's first
  const long long wk0 = f0 / span;
  const int np = static_cast<int>((f1 - 1) / span - wk0) + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int rows, x0;                                  // the tile's rows, its first packed row
  if (ROWS > 0) {
    x0 = w.rt * TILE_ROWS;
    rows = min(TILE_ROWS, w.s.nq * p.G - x0);
  } else {
    x0 = w.rt * tpi * p.G;
    rows = min(tpi, w.s.nq - w.rt * tpi) * p.G;
  }
  // rows of whole-token tiles stand 128 / G tokens to each 128
  const int per128 = (128 / p.G > 0 ? 128 / p.G : 1) * p.G;
  // a piece's place: the item's first piece is its worker's second slot unless the span begins with it
  auto place = [&](int i, int r) -> long long {
    return ((wk0 + i) * 2 + (i == 0 && f0 != wk0 * span ? 1 : 0)) * TILE_ROWS +
           (ROWS > 0 ? r : r + r / per128 * (128 - per128));
  };
  auto finish = [&](int r, float m, float l, const float (&acc)[V]) {
    const int x = x0 + r, t = x / p.G, head = w.h * p.G + x - t * p.G;
    const long long row = static_cast<long long>(w.s.q0 + t) * p.hq + head;
    const long long li = static_cast<long long>(head) * p.n_tokens + w.s.q0 + t;
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
  if (np <= 2 * NW) {
    for (int r = blockIdx.y * NW + warp; r < rows; r += gridDim.y * NW) {
      gather(r, 0, 1, m, l, acc);
      finish(r, m, l, acc);
    }
    return;
  }
  for (int r = blockIdx.y; r < rows; r += gridDim.y) {
    gather(r, warp, NW, m, l, acc);
    float *mine = red + warp * (D + 4);
#pragma unroll
    for (int c = 0; c < V; ++c) mine[lane * V + c] = acc[c];
    if (lane == 0) {
      mine[D] = m;
      mine[D + 1] = l;
    }
    __syncthreads();
    if (warp == 0) {
      float mt = -INFINITY, lt = 0.f;
#pragma unroll
      for (int k = 0; k < NW; ++k) mt = fmaxf(mt, red[k * (D + 4) + D]);
      const float mb = mt == -INFINITY ? 0.f : mt;
#pragma unroll
      for (int c = 0; c < V; ++c) acc[c] = 0.f;
#pragma unroll
      for (int k = 0; k < NW; ++k) {
        const float f = exp2f(red[k * (D + 4) + D] - mb);
        lt += f * red[k * (D + 4) + D + 1];
#pragma unroll
        for (int c = 0; c < V; ++c) acc[c] = fmaf(f, red[k * (D + 4) + lane * V + c], acc[c]);
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

template <int D>
inline size_t join_smem_bytes(int n_seqs, bool infos) {
  return 80 + 8 * (D + 4) * 4 + 8ull * (n_seqs + 1) + (infos ? sizeof(SeqInfo) * n_seqs : 0);
}



}  // namespace attn
