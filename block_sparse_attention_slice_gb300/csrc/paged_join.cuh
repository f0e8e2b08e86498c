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
  static constexpr int V = D / 32, BATCH = 4;
  float m = -INFINITY, l = 0.f, acc[V];
  __device__ __forceinline__ Gather() {
#pragma unroll
    for (int c = 0; c < V; ++c) acc[c] = 0.f;
  }
  // Sets the sum of n <= 4 pieces: every lane reads their (m, l) itself, all
  // loads at once, and no shuffle is needed.
  template <typename FO, typename FM>
  __device__ __forceinline__ void few(int n, FO o_of, FM ml_of) {
    const int lane = threadIdx.x & 31;
    float2 ml[4];
    float y[4][V];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k < n) {
        ml[k] = *reinterpret_cast<const float2 *>(ml_of(k));
        const float *src = o_of(k) + lane * V;
        if constexpr (V == 4) {
          const float4 z = *reinterpret_cast<const float4 *>(src);
          y[k][0] = z.x, y[k][1] = z.y, y[k][2] = z.z, y[k][3] = z.w;
        } else {
          const float2 z = *reinterpret_cast<const float2 *>(src);
          y[k][0] = z.x, y[k][1] = z.y;
        }
      }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k < n) m = fmaxf(m, ml[k].x);
    const float mb = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k < n) {
        const float f = exp2f(ml[k].x - mb);
        l = fmaf(f, ml[k].y, l);
#pragma unroll
        for (int c = 0; c < V; ++c) acc[c] = fmaf(f, y[k][c], acc[c]);
      }
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
// Bound by L2 and latency: its pieces were written just before.  12 us behind
// 152 spans of 256 rows (38 MB of pieces), 3 us behind a single sequence.
// PACKED: rows stand as they are counted; else 128 / G whole tokens to each
// 128 rows.
template <int D, int TILE_ROWS, bool PACKED>
__global__ void __launch_bounds__(256, 4) paged_join_kernel(const PagedParams p) {
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
  if (np <= 4) {
    for (int r = blockIdx.y * NW + warp; r < cut.rows; r += gridDim.y * NW) {
      Gather<D> g;
      g.few(np, [&](int k) { return p.part_o + place(k, r) * D; }, [&](int k) { return p.part_ml + place(k, r) * 2; });
      finish(r, g.m, g.l, g.acc);
    }
    return;
  }
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

// The largest i < n with a[i] <= x, where a does not decrease; 0 if there is none.
__device__ __forceinline__ int last_not_above(const int32_t *a, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(a + mid) <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Whether a record names pieces that the pass has.
__device__ __forceinline__ bool in_bounds(const Rec4 &r, const PagedParams &p, int rows) {
  const long long workers = static_cast<long long>(p.n_spans) * p.hp;
  return r.np <= 0 || (r.np <= p.n_spans && r.worker >= 0 && r.worker + (r.np - 1ll) * p.hp < workers && (r.slot0 & ~1) == 0 &&
                       r.row >= 0 && r.row < rows);
}

// Merges what two passes over the same rows left, the prefix's and that of
// what follows it: a warp a row.  A row's records were written in this call
// exactly if the row belongs to a sequence (and to a group), which is looked
// up here, while the passes still run, rather than having the records cleared
// before them.  9 us for 8192 rows of 128 columns, 7 for 6400 of 64.
template <int D>
__global__ void __launch_bounds__(256, 4) paged_join_pair_kernel(const PagedParams pre, const PagedParams p,
                                                                 const int pre_rows, const int rows) {
  constexpr int V = D / 32;
  admit_next();
  const int lane = threadIdx.x & 31;
  const long long row = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int t = static_cast<int>(row / p.hq);
  bool mine = false, grouped = false;
  if (t < p.n_tokens) {
    const int b = p.q_ptr ? last_not_above(p.q_ptr, p.n_seqs, t) : t;
    const SeqInfo s = seq_info(p, b);
    mine = t >= s.q0 && t < s.q0 + s.nq;
    const SeqInfo g = seq_info(pre, last_not_above(pre.group_ptr, pre.n_seqs, b));
    grouped = t >= g.q0 && t < g.q0 + g.nq;
  }
  after_previous();
  if (!mine) return;                               // of no sequence: left as it is
  Rec4 a{0, 0, REC_EMPTY, 0}, b = p.rec[row];
  if (grouped) a = pre.rec[row];
  // a pass that gave up (a bounded wait ran out) left some records unwritten
  if (!in_bounds(a, pre, pre_rows)) a.np = REC_EMPTY;
  if (!in_bounds(b, p, rows)) b.np = REC_EMPTY;
  const int na = a.np < 0 ? 0 : a.np ? a.np : 1, nb = b.np < 0 ? 0 : b.np ? b.np : 1, np = na + nb;
  // row of piece i in its pass's pieces, or (np = 0) in the dense arrays
  auto place = [&](int i, bool &first, bool &dense) -> long long {
    first = i < na;
    const Rec4 &r = first ? a : b;
    const int k = first ? i : i - na;
    dense = r.np == 0;
    if (dense) return row;
    return ((static_cast<long long>(r.worker) + k * (first ? pre.hp : p.hp)) * 2 + (k == 0 ? r.slot0 : 0)) *
               (first ? pre_rows : rows) + r.row;
  };
  Gather<D> g;
  for (int base = 0; base < np; base += 32) {
    float2 ml = make_float2(-INFINITY, 0.f);
    if (base + lane < np) {
      bool first, dense;
      const long long at = place(base + lane, first, dense);
      const PagedParams &x = first ? pre : p;
      ml = *reinterpret_cast<const float2 *>((dense ? x.dense_ml : x.part_ml) + at * 2);
    }
    g.add(min(32, np - base), ml, [&](int k) -> const float * {
      bool first, dense;
      const long long at = place(base + k, first, dense);
      const PagedParams &x = first ? pre : p;
      return (dense ? x.dense_o : x.part_o) + at * D;
    });
  }
  float fo, lse;
  row_final(g.m, g.l, fo, lse);
#pragma unroll
  for (int c = 0; c < V; c += 2) store_pair<D>(p, row, lane * V + c, g.acc[c] * fo, g.acc[c + 1] * fo);
  if (lane == 0) p.lse[(row - static_cast<long long>(t) * p.hq) * p.n_tokens + t] = lse;
}

}  // namespace attn
