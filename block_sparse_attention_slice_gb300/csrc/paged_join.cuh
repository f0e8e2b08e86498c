// Joining the pieces of the items that cross span boundaries.
#pragma once
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "launch.cuh"
#include "paged_plan.cuh"

namespace attn {

// A running summary over pieces, held by one warp: lane's V columns of O.
template <int D>
struct Gather {
  static constexpr int V = D / 32, BATCH = 8;
  float m = -INFINITY, l = 0.f, acc[V];
  __device__ __forceinline__ Gather() {
#pragma unroll
    for (int c = 0; c < V; ++c) acc[c] = 0.f;
  }
  // Adds n <= 32 pieces in order; o_of(i) is the address of piece i's O row,
  // and lane i has its (m, l).  The first rows are requested before the
  // weights that they wait for are known.
  template <typename F>
  __device__ __forceinline__ void add(int n, float2 ml, F o_of) {
    const int lane = threadIdx.x & 31;
    float y[BATCH][V];
    auto fetch = [&](int k0) {
#pragma unroll
      for (int k = 0; k < BATCH; ++k)
        if (k0 + k < n) {
          const float *src = o_of(k0 + k) + lane * V;
          if constexpr (V == 4) {
            const float4 z = *reinterpret_cast<const float4 *>(src);
            y[k][0] = z.x, y[k][1] = z.y, y[k][2] = z.z, y[k][3] = z.w;
          } else {
            const float2 z = *reinterpret_cast<const float2 *>(src);
            y[k][0] = z.x, y[k][1] = z.y;
          }
        }
    };
    fetch(0);
    float top = lane < n ? ml.x : -INFINITY;
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    top = fmaxf(top, m);
    const float mb = top == -INFINITY ? 0.f : top, old = exp2f(m - mb);
    const float f = lane < n ? exp2f(ml.x - mb) : 0.f;
    float s = lane < n ? f * ml.y : 0.f;
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    m = top;
    l = l * old + s;
#pragma unroll
    for (int c = 0; c < V; ++c) acc[c] *= old;
    for (int k0 = 0; k0 < n; k0 += BATCH) {
      if (k0) fetch(k0);
#pragma unroll
      for (int k = 0; k < BATCH; ++k) {
        const float g = __shfl_sync(0xffffffffu, f, (k0 + k) & 31);
        if (k0 + k < n) {
#pragma unroll
          for (int c = 0; c < V; ++c) acc[c] = fmaf(g, y[k][c], acc[c]);
        }
      }
    }
  }
};

// Merges the pieces of the items that cross span boundaries: block x looks at
// what worker x left and, where an item begins there and goes on, merges that
// item's rows (blockIdx.y of gridDim.y takes its part of them).  Few pieces:
// one warp a row.  Many (a long sequence alone in the batch): the block's
// warps share a row's pieces and add their sums.  Pieces are added in a fixed
// order, so results do not vary from run to run.
// PACKED: rows stand as they are counted; else 128 / G whole tokens to each
// 128 rows.
template <int D, int TILE_ROWS, bool PACKED>
__global__ void __launch_bounds__(256) paged_join_kernel(const PagedParams p) {
  constexpr int NW = 8, V = D / 32;
  __shared__ float red[NW][D + 4];
  admit_next();
  after_previous();
  const Cut cut = p.cuts[blockIdx.x];
  if (cut.rows == 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, np = cut.np;
  const int per128 = PACKED ? 128 : 128 / p.G * p.G;
  auto place = [&](int i, int r) -> long long {
    return ((static_cast<long long>(blockIdx.x) + i * p.hp) * 2 + (i == 0 ? cut.slot0 : 0)) * TILE_ROWS +
           (PACKED ? r : r + r / per128 * (128 - per128));
  };
  auto finish = [&](int r, float m, float l, const float (&acc)[V]) {
    const int x = cut.x0 + r, t = x / p.G, head = cut.h * p.G + x - t * p.G;
    const long long row = static_cast<long long>(cut.q0 + t) * p.hq + head;
    float fo, lse;
    row_final(m, l, fo, lse);
#pragma unroll
    for (int c = 0; c < V; c += 2) store_pair<D>(p, row, lane * V + c, acc[c] * fo, acc[c + 1] * fo);
    if (lane == 0) p.lse[static_cast<long long>(head) * p.n_tokens + cut.q0 + t] = lse;
  };
  // pieces i0, i0 + step, ... of row r
  auto gather = [&](Gather<D> &g, int r, int i0, int step) {
    for (int base = i0; base < np; base += 32 * step) {
      const int n = min(32, (np - base + step - 1) / step);
      float2 ml = make_float2(-INFINITY, 0.f);
      if (lane < n) ml = *reinterpret_cast<const float2 *>(p.part_ml + place(base + lane * step, r) * 2);
      g.add(n, ml, [&](int k) { return p.part_o + place(base + k * step, r) * D; });
    }
  };
  if (np <= NW) {
    for (int r = blockIdx.y * NW + warp; r < cut.rows; r += gridDim.y * NW) {
      Gather<D> g;
      gather(g, r, 0, 1);
      finish(r, g.m, g.l, g.acc);
    }
    return;
  }
  for (int r = blockIdx.y; r < cut.rows; r += gridDim.y) {
    Gather<D> g;
    gather(g, r, warp, NW);
#pragma unroll
    for (int c = 0; c < V; ++c) red[warp][lane * V + c] = g.acc[c];
    if (lane == 0) {
      red[warp][D] = g.m;
      red[warp][D + 1] = g.l;
    }
    __syncthreads();
    if (warp == 0) {
      Gather<D> all;
      const float2 ml = lane < NW ? make_float2(red[lane][D], red[lane][D + 1]) : make_float2(-INFINITY, 0.f);
      all.add(NW, ml, [&](int k) -> const float * { return red[k]; });
      finish(r, all.m, all.l, all.acc);
    }
    __syncthreads();
  }
}

// Merges the pieces of two passes over the same rows: a warp a row.
struct JoinPair {
  const Rec4 *rec[2];
  const float *dense_o[2], *dense_ml[2], *part_o[2], *part_ml[2];
  int tile_rows[2], hp[2];
};
template <int D>
__global__ void __launch_bounds__(256) paged_join_pair_kernel(const PagedParams p, const JoinPair q) {
  constexpr int V = D / 32;
  admit_next();
  after_previous();
  const int lane = threadIdx.x & 31;
  const long long row = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (row >= static_cast<long long>(p.n_tokens) * p.hq) return;
  const Rec4 a = q.rec[0][row], b = q.rec[1][row];
  if (b.np == -1) return;                          // of no sequence: left as it is
  const int na = a.np < 0 ? 0 : a.np ? a.np : 1, nb = b.np < 0 ? 0 : b.np ? b.np : 1, np = na + nb;
  // row of piece i in its pass's pieces, or (np = 0) in the dense arrays
  auto place = [&](int i, int &x, bool &dense) -> long long {
    x = i < na ? 0 : 1;
    const Rec4 &r = x ? b : a;
    const int k = x ? i - na : i;
    dense = r.np == 0;
    if (dense) return row;
    return ((static_cast<long long>(r.worker) + k * q.hp[x]) * 2 + (k == 0 ? r.slot0 : 0)) * q.tile_rows[x] + r.row;
  };
  Gather<D> g;
  for (int base = 0; base < np; base += 32) {
    float2 ml = make_float2(-INFINITY, 0.f);
    if (base + lane < np) {
      int x;
      bool dense;
      const long long at = place(base + lane, x, dense);
      ml = *reinterpret_cast<const float2 *>((dense ? q.dense_ml[x] : q.part_ml[x]) + at * 2);
    }
    g.add(min(32, np - base), ml, [&](int k) -> const float * {
      int x;
      bool dense;
      const long long at = place(base + k, x, dense);
      return (dense ? q.dense_o[x] : q.part_o[x]) + at * D;
    });
  }
  float fo, lse;
  row_final(g.m, g.l, fo, lse);
#pragma unroll
  for (int c = 0; c < V; c += 2) store_pair<D>(p, row, lane * V + c, g.acc[c] * fo, g.acc[c + 1] * fo);
  if (lane == 0) p.lse[row % p.hq * p.n_tokens + row / p.hq] = lse;
}

}  // namespace attn
